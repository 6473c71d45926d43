"""How long a 4-bit attention call takes whose waits run out: the limit of a wait (20 ms in the test's entry point), and once more for
the copies that may be under way, however many entries a ring has (3 to 12 here)."""
import time

import pytest

torch = pytest.importorskip("torch")

import w4a8_verify_gb300 as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    W.lib()


@pytest.mark.parametrize("n,D,P", [(1, 128, 1200), (4, 64, 500), (16, 64, 500), (16, 128, 500)])
def test_time_of_a_call_whose_waits_run_out(n, D, P):
    S, H, G = 2, 8, 4
    cache = W.KV4Cache(S, H, D, P)
    cache.tensors["pages"].zero_()
    cache.len.fill_(64 * P)
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    q = torch.randn((S, n, H * G, D), generator=g, device="cuda")
    want = cache.attention(q)
    torch.cuda.synchronize()
    real, ms = cache._attention, []
    try:
        cache._attention = lambda c, a, w, b, st: W.lib().w4a8_kv4_attention_inject_timeout(c, a, w, b, 3, st)
        for _ in range(3):
            begin = time.perf_counter()
            got = cache.attention(q)
            torch.cuda.synchronize()
            ms.append((time.perf_counter() - begin) * 1e3)
    finally:
        cache._attention = real
    assert cache.check() == W.FLAG_ERR_TIMEOUT
    assert torch.isnan(got).any() and not torch.isnan(got).all()
    assert 20 <= min(ms) < 60, ms                                    # with a limit for each entry: 84, 266, 103, 103
    cache.tensors["ctl"].zero_()
    assert torch.equal(cache.attention(q), want) and cache.check() == 0
