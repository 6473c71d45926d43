"""Appends of a few rows to caches of few and of many heads: whichever kernel takes them, every code and scale is the definition's
(oracle/kv4.py), and nothing else of the pages changes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_verify_gb300 as W
from oracle import kv4 as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    W.lib()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("S,H,D,n", [
    (2, 4, 64, 16),                                                  # a tile to a warp
    (1, 8, 128, 1), (1, 8, 128, 9), (1, 33, 64, 1), (3, 40, 64, 16), (1, 1024, 64, 2),   # heads and lengths apart
    (40, 16, 64, 1), (70, 16, 64, 5), (160, 8, 64, 16),              # several tiles to a warp
])
def test_appended_rows(S, H, D, n, dtype):
    rng = np.random.default_rng(S * H + n)
    g = torch.Generator(device="cuda")
    g.manual_seed(S + H)
    P = 3
    cache = W.KV4Cache(S, H, D, P)
    cache.tensors["pages"].random_(0, 180, generator=g)              # any codes, finite scales
    cache.tensors["table"].copy_(torch.randperm(S * P, generator=g, device="cuda").view(S, P).to(torch.int32))
    lens = rng.integers(0, 64 * P - 2 * n, S)
    lens[0], lens[-1] = 64 * P - 2 * n, 63
    cache.len.copy_(torch.from_numpy(lens.astype(np.int32)))
    first = torch.zeros(S, dtype=torch.int32, device="cuda")
    full = torch.full((S,), 64 * P, dtype=torch.int32, device="cuda")
    want = [x.cpu().numpy() for x in cache.read(first, 64 * P, length=full)]
    for index in (False, True):
        x = [(torch.randn((S, n, H, D), generator=g, device="cuda") * a) for a in (1.0, 3.0)]
        x = [a.to(dtype) for a in x]
        counts = rng.integers(0, n + 1, S)
        counts[0] = n
        order = rng.integers(0, n, (S, n)) if index else np.tile(np.arange(n), (S, 1))
        cache.append(*x, counts=torch.from_numpy(counts.astype(np.int32)).cuda(),
                     index=torch.from_numpy(order.astype(np.int32)).cuda() if index else None)
        for i in range(2):
            codes, scales = O.quantize(x[i].float().cpu().numpy())
            rows = O.value(codes, scales).astype(np.float32)
            for s in range(S):
                want[i][s, lens[s]:lens[s] + counts[s]] = rows[s, order[s, :counts[s]]]
        lens = lens + counts
        assert cache.len.tolist() == lens.tolist()
        for got, w in zip(cache.read(first, 64 * P, length=full), want):
            assert np.array_equal(got.cpu().numpy(), w)
    assert cache.check() == 0
