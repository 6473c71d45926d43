"""A pool of fewer pages than its sequences have room for, as a reset leaves it: no page has two owners, and what needs a page that no
sequence was given is left out and reported."""
import pytest

torch = pytest.importorskip("torch")

import w4a8_verify_gb300 as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    W.lib()


@pytest.mark.parametrize("n_pages", [1, 7, 12, 20])
def test_pages_of_a_small_pool_have_one_owner(n_pages):
    S, H, D, P = 3, 2, 64, 4
    cache = W.KV4Cache(S, H, D, P, n_pages)
    cache.tensors["pages"].fill_(255)
    want = torch.arange(S * P, device="cuda")
    want[n_pages:] = -1
    assert torch.equal(cache.tensors["table"].view(-1).long(), want)
    g = torch.Generator(device="cuda")
    g.manual_seed(n_pages)
    x = torch.randn((S, 64 * P, H, D), generator=g, device="cuda")
    roomy = W.KV4Cache(S, H, D, P)
    for c in (cache, roomy):
        c.append(x[:, :200], x[:, :200])
        c.append(x[:, 200:], x[:, 200:])
    first = torch.zeros(S, dtype=torch.int32, device="cuda")
    for got, full in zip(cache.read(first, 64 * P), roomy.read(first, 64 * P)):
        there = (want >= 0).view(S, P, 1, 1, 1)
        assert torch.equal(got, torch.where(there, full.view(S, P, 64, H, D), 0.0).view_as(got))
    assert cache.check() == (W.FLAG_ERR_TREE if n_pages < S * P else 0)
    # the pages that there are, dealt anew
    cache.reset()
    if n_pages >= 6:
        cache.tensors["table"][:, :2] = torch.arange(6, device="cuda", dtype=torch.int32).view(3, 2).flip(0)
        cache.append(x[:, :128], x[:, :128])
        assert all(torch.equal(a, b[:, :128]) for a, b in zip(cache.read(first, 128), roomy.read(first, 128))) and cache.check() == 0
