"""4-bit attention with logits up to the documented 2^20 in magnitude, all close to one another, in every order of pages: weights stay
in the range of their f16 form.

All keys share a large part, 7 a s of dim 0; dim 32, with a scale of its own, sets them apart by up to 16 in log2.  A logit of L is
rounded to fp32 (2^-24 L) when it is scaled and again when the maximum is taken off; with q's f16 terms (2^-23 of its largest, times
7 s) that is at most 2^-22 L in all, 1/4 at 2^20: weights are off by a factor of 2^(2 log2(e) / 4) = 1.65 or its inverse at most, so an
output lies between the values' ends, and the definition's weights w give sum w v / 1.65^2 <= out <= 1.65^2 sum w v for values above 0.
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


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,G", [(1, 4), (1, 12), (20, 4)])          # one and two column tiles, tcgen05
def test_large_logits_close_to_one_another(n, G, dtype, sign):
    H, D, P = 2, 64, 60
    g = torch.Generator(device="cuda")
    g.manual_seed(n + G)
    # code of dim 32 per page: down, up by more and by less than the slack of 8, and at random
    step = torch.tensor([0, 7, 0, -7, 0, 3, 7, -2, 1, 5, 6, 7, -7, 4, 0], device="cuda").repeat_interleave(64)
    code = torch.cat([step, torch.randint(-7, 8, (64 * (P - 15),), generator=g, device="cuda")]).float()
    k = torch.zeros(1, 64 * P, H, D, device="cuda")
    k[..., 0] = 7.0                                                  # scale 1
    k[..., 32] = code[None, :, None] / 8                             # scale 1/8
    k[..., 33] = 7.0 / 8
    v = torch.rand((1, 64 * P, H, D), generator=g, device="cuda") + 0.5
    cache = W.KV4Cache(1, H, D, P)
    cache.append(k, v)
    kc, vc = (x[0].double() for x in cache.read(torch.zeros(1, dtype=torch.int32, device="cuda"), 64 * P))
    assert torch.equal(kc, k[0].double())
    for large in (0.0, 1e3, 2.0 ** 16, 2.0 ** 20 - 64):
        q = torch.zeros(1, n, H * G, D, device="cuda")
        q[..., 0] = large / 7
        # codes -7 .. 7 are -8 .. 8 in log2 apart
        q[..., 32] = 8 / 1.4426950408889634 / (7 / 8)
        q = (q * sign).to(dtype)
        out = cache.attention(q, scale=float(sign)).double()
        assert torch.isfinite(out).all(), large
        w = torch.softmax(torch.einsum("nhd,thd->hnt", (q[0, :, ::G].double() * sign), kc), -1)
        ref = torch.einsum("hnt,thd->nhd", w, vc).repeat_interleave(G, dim=1)
        most = 1.65 ** (2 * large / 2.0 ** 20) * (1 + 2.0 ** -7)
        assert (out[0] <= ref * most).all() and (out[0] >= ref / most).all(), large
    assert cache.check() == 0
