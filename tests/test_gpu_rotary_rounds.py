"""The rotation where a warp goes through several rounds of a token's heads (many tokens): queries and keys in one warp, a last
share that is not full, in place, rows that are not 16-byte aligned.

Sampled tokens against the definition in 64 bits, with the bound derived in tests/test_gpu_rotary.py: 2^-19 of the turned pair's
size, and half a step (2^-8) of bf16 outputs.  All tokens against calls of a few of them, whose warps have one round each: the
same arithmetic, so the same bits.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import w4a8_verify_gb300 as W
from oracle import rotary as R

pytestmark = pytest.mark.gpu
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    W.lib()


def _rounds(tokens, heads, D):
    """Rounds of a token, of a warp: the kernel's rule (152 x 16 warps to be kept busy)."""
    per = 8 if D <= 64 else 4 if D <= 128 else 2
    rounds = -(-heads // per)
    return rounds, min(rounds, -(-tokens * rounds // (152 * 16)))


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("D,Hq,Hk,n,neighbours,rot", [
    (128, 32, 8, 700, False, 128),
    (128, 9, 2, 700, True, 64),
    (64, 32, 8, 700, False, 64),
    (256, 9, 2, 700, False, 128),
    (80, 21, 1, 1900, False, 80),
    (128, 32, 8, 5001, False, 128),
])
def test_rounds_of_a_warp(D, Hq, Hk, n, neighbours, rot, dtype, aligned):
    rng = np.random.default_rng(D + n)
    S = 2
    rounds, iters = _rounds(S * n, Hq + Hk, D)
    assert iters > 1                                                # what this test is for
    g = torch.Generator(device="cuda")
    g.manual_seed(D)
    base = torch.randn((S, n, Hq + 2 * Hk, D), generator=g, device="cuda").to(TYPES[dtype])
    if not aligned:
        x = torch.empty(S, n, Hq + 2 * Hk, D + 1, dtype=base.dtype, device="cuda")[..., 1:]
        x.copy_(base)
    else:
        x = base.clone()
    gains = [(1 + 0.3 * rng.standard_normal(D)).astype(np.float32) for _ in range(2)]
    gq, gk = (torch.from_numpy(a).cuda() for a in gains)
    pos = torch.randint(0, 60000, (S, n), generator=g, device="cuda", dtype=torch.int32)
    start = torch.tensor([3, 70000], dtype=torch.int32, device="cuda")
    counts = torch.tensor([n, n - 77], dtype=torch.int32, device="cuda")
    rope = W.Rotary(D, rot, neighbours=neighbours)
    kw = dict(start=start, eps=1e-5, q_gain=gq, k_gain=gk)
    q, k = rope.apply(x[:, :, :Hq], x[:, :, Hq:Hq + Hk], positions=pos, **kw)
    # in place, padded
    a, b = x[:, :, :Hq], x[:, :, Hq:Hq + Hk]
    rope.apply(a, b, positions=pos, counts=counts, q_out=a, k_out=b, **kw)
    assert torch.equal(x[0, :, :Hq], q[0]) and torch.equal(x[0, :, Hq:Hq + Hk], k[0])
    assert torch.equal(x[1, :n - 77, :Hq], q[1, :n - 77]) and torch.equal(x[1, :n - 77, Hq:Hq + Hk], k[1, :n - 77])
    assert torch.equal(x[1, n - 77:], base[1, n - 77:]) and torch.equal(x[:, :, Hq + Hk:], base[:, :, Hq + Hk:])
    # a few tokens to a call: one round to a warp
    few = (152 * 16) // (2 * rounds)
    assert _rounds(S * few, Hq + Hk, D)[1] == 1
    for at in range(0, n, few):
        part = slice(at, min(n, at + few))
        q1, k1 = rope.apply(base[:, part, :Hq].contiguous(), base[:, part, Hq:Hq + Hk].contiguous(),
                            positions=pos[:, part].contiguous(), **kw)
        assert torch.equal(q1, q[:, part]) and torch.equal(k1, k[:, part]), at
    inv = 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    for s, j in [(0, 0), (1, n - 1)] + [(int(rng.integers(S)), int(rng.integers(n))) for _ in range(6)]:
        angle = np.full(rot // 2, float(int(start[s]) + int(pos[s, j])))
        for heads, y, gain, at in ((Hq, q, gains[0], 0), (Hk, k, gains[1], Hq)):
            for h in sorted({0, heads - 1, heads // 2}):
                xn = base[s, j, at + h].double().cpu().numpy()
                want = R.turn(xn, angle, inv, neighbours, 1.0, 1e-5, gain)
                size = R.turn(xn, [], [], False, 1.0, 1e-5, gain)
                i0, i1 = (slice(0, rot, 2), slice(1, rot, 2)) if neighbours else (slice(0, rot // 2), slice(rot // 2, rot))
                both = np.hypot(size[i0], size[i1])
                size = np.abs(size)
                size[i0], size[i1] = both, both
                bound = 2.0 ** -19 * size + (2.0 ** -8 * np.abs(want) if dtype == "bf16" else 0)
                err = np.abs(y[s, j, h].double().cpu().numpy() - want)
                assert (err <= bound + 1e-38).all(), (s, j, at + h, (err / (bound + 1e-38)).max())
