"""The sums of 4-bit attention over the longest caches: a million tokens to a sequence, one warp pair to each (sequence, KV head), whose
sequences share one sequence's pages.

Each dim of the values is the same number v for all tokens, so the definition's output is v whatever the weights.  v is c s, seven
bits, exact in bf16 and fp32.  bf16: the weights' f16 factors are off by 2^-11 of them, the output's rounding by 2^-8 of it.  fp32:
the bound derived in tests/test_gpu_kv4.py without logits to be off, 2^-16.  The sums themselves are of up to 2^15 parts of a
warp in fp32, whose roundings to nearest go either way: sqrt(2^15) 2^-24 is below 2^-16.
"""
import pytest

torch = pytest.importorskip("torch")

import w4a8_verify_gb300 as W

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    W.lib()


@pytest.fixture(scope="module")
def pool():
    """A sequence of 16384 full pages, 2 heads of 128, and what its values are."""
    P, H, D = 16384, 2, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    one = W.KV4Cache(1, H, D, P)
    v = torch.rand((1, 1, H, D), generator=g, device="cuda") + 0.5
    for _ in range(P // 1024):
        k = torch.randn((1, 65536, H, D), generator=g, device="cuda") * 0.3
        one.append(k, v.expand(1, 65536, H, D))
    assert one.check() == 0 and one.len.item() == 64 * P
    return one, one.read(torch.zeros(1, dtype=torch.int32, device="cuda"), 64)[1][0, 0].double()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("S,G", [(608, 4), (304, 12)])               # one and two column tiles
def test_values_of_a_million_tokens(pool, S, G, dtype):
    one, v = pool
    _, H, D, P, _ = one.shape
    cache = W.KV4Cache(S, H, D, P, P, tensors=dict(
        one.tensors, table=one.tensors["table"].expand(S, P).contiguous(), len=one.len.expand(S).contiguous()))
    g = torch.Generator(device="cuda")
    g.manual_seed(G)
    q = torch.randn((S, 1, H * G, D), generator=g, device="cuda").to(dtype)
    out = cache.attention(q, scale=D ** -0.5).double().view(S, H, G, D)
    off = (out / v[:, None] - 1).abs().max().item()
    assert off <= (2.0 ** -11 + 2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -16), off
    assert cache.check() == 0
