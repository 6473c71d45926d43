"""The 4-bit key/value cache by definition: groups of 32 dims, the bytes of a page, and attention over it.

A cache here is a list of rows per sequence with their codes and scales written out; the bytes of a page follow the
formulas of include/w4a8.h one at a time.  Scales and codes are decided in fp32, the precision of the kernels; everything
else is fp64.
"""
from __future__ import annotations

import numpy as np

PAGE, GROUP, NAN_BYTE = 64, 32, 255


def scale_value(byte):
    """Value of a scale byte (fp64)."""
    if byte == NAN_BYTE:
        return np.nan
    e, m = byte >> 3, byte & 7
    return m * 2.0 ** -17 if e == 0 else (8 + m) * 2.0 ** (e - 18)


VALUES = np.array([scale_value(b) for b in range(184)])   # ascending; 183 is 240


def quantize(x):
    """fp32 [..., D] -> (codes int [..., D], scale bytes int [..., D / 32])."""
    x = np.asarray(x, dtype=np.float32)
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    finite = np.isfinite(g).all(axis=-1)
    s = (np.abs(np.where(finite[..., None], g, 0)).max(axis=-1) / np.float32(7)).astype(np.float64)
    # the nearest value; halfway between two: the even byte
    hi = np.minimum(np.searchsorted(VALUES, s), len(VALUES) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = VALUES[hi] - s, s - VALUES[lo]
    byte = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    byte = np.where(s >= VALUES[-1], len(VALUES) - 1, byte)
    scale = VALUES[byte].astype(np.float32)[..., None]
    with np.errstate(over="ignore", invalid="ignore"):
        q = (g / np.where(scale > 0, scale, 1)).astype(np.float32)
        code = np.clip(np.rint(q), -7, 7)
    code = np.where((scale > 0) & finite[..., None], code, 0).astype(np.int64)
    return code.reshape(x.shape), np.where(finite, byte, NAN_BYTE)


def value(codes, bytes_):
    """fp64 values of codes [..., D] with scale bytes [..., D / 32]."""
    s = np.vectorize(scale_value, otypes=[np.float64])(bytes_)
    return codes * np.repeat(s, GROUP, axis=-1)


def key_place(D, tok, d):
    """(16-bit word, field) of a key's code in a page, byte of its scale."""
    word = (((tok // 16 * (D // 64) + d // 64) * 32 + tok % 8 * 4 + d % 32 // 8) * 4 + d % 64 // 32 * 2 + d % 8 // 4) * 2 + d % 2
    return word, d % 4 // 2 * 2 + tok % 16 // 8, 64 * D + (tok // 16 * 8 + tok % 8) * (D // 16) + tok % 16 // 8 * (D // 32) + d // 32


def value_place(D, tok, d):
    word = (((tok // 16 * (D // 64) + d // 64) * 32 + d % 8 * 4 + tok % 8 // 2) * 4 + d % 64 // 16) * 2 + tok % 2
    return (16 * D + word, d % 16 // 8 * 2 + tok % 16 // 8,
            66 * D + ((tok // 16 * 4 + tok % 8 // 2) * (D // 32) + d // 32) * 4 + tok % 16 // 8 * 2 + tok % 2)


def read_page(page, D, place):
    """Bytes [68 D] of a page of one head -> (codes [64][D], scale bytes [64][D / 32])."""
    tok, d = np.meshgrid(np.arange(PAGE), np.arange(D), indexing="ij")
    word, field, scale = place(D, tok, d)
    w = page[2 * word].astype(np.uint32) | page[2 * word + 1].astype(np.uint32) << 8
    w = (w >> 2) | (w << 14 & 0xffff)                     # turned back
    return (w >> (4 * field).astype(np.uint32) & 15).astype(np.int64) - 8, page[scale][:, ::GROUP].astype(np.int64)


class Cache:
    """Rows of S sequences: ``rows[s]`` is (key codes, key scales, value codes, value scales), each [length][H][..]."""

    def __init__(self, S, H, D):
        self.S, self.H, self.D = S, H, D
        none = lambda w: np.zeros((0, H, w), np.int64)  # noqa: E731
        self.rows = [(none(D), none(D // GROUP), none(D), none(D // GROUP)) for _ in range(S)]

    def length(self, s):
        return len(self.rows[s][0])

    def append(self, s, k, v):
        """Rows k, v fp32 [n][H][D] of sequence s."""
        self.rows[s] = tuple(np.concatenate([a, b]) for a, b in zip(self.rows[s], quantize(k) + quantize(v)))

    def held(self, s, h):
        """fp64 keys and values [tokens][D]."""
        kc, ks, vc, vs = self.rows[s]
        return value(kc[:, h], ks[:, h]), value(vc[:, h], vs[:, h])


def attention(k, v, q, k_new, v_new, mask, scale):
    """One query row q fp64 [D] over held rows k, v and the new rows it sees (bits of mask): (out [D], scale times the largest
    |q_d| times the largest sum_d |k_d|)."""
    sees = [j for j in range(len(k_new)) if mask >> j & 1]
    D = len(q)
    k = np.concatenate([k, np.asarray(k_new, np.float64)[sees].reshape(-1, D)])
    v = np.concatenate([v, np.asarray(v_new, np.float64)[sees].reshape(-1, D)])
    if not len(k):
        return np.zeros(D), 0.0
    logits = k @ q * scale
    e = np.exp(logits - logits.max())
    return (e / e.sum()) @ v, float(np.abs(k).sum(axis=1).max() * np.abs(q).max() * abs(scale))
