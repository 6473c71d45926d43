"""The 8-bit key/value cache by definition: pages, attention over them, page selection and eviction.

A cache here is a list of positions per (sequence, KV head) with their page codes written out; the bytes of a
page follow the formulas of include/w4a8.h one at a time.  Codes and scores, which decide integers, are taken in
fp32, the precision of the kernels; everything else is fp64.
"""
from __future__ import annotations

import numpy as np

PAGE = 64


def quantize_page(x):
    """fp32 [64][D] -> (codes int [64][D], fp32 scale); not finite -> codes 0, scale NaN."""
    x = np.asarray(x, dtype=np.float32)
    if not np.isfinite(x).all():
        return np.zeros(x.shape, dtype=np.int64), np.float32(np.nan)
    s = np.float32(np.abs(x).max()) / np.float32(127)
    if not s > 0:
        return np.zeros(x.shape, dtype=np.int64), np.float32(0)
    return np.clip(np.rint((x / s).astype(np.float32)), -127, 127).astype(np.int64), s


def key_byte(D, tok, d):
    return (((((tok // 16 * (D // 32) + d // 32) * 8 + tok % 8) * 4 + d % 32 // 8) * 2 + d % 8 // 4) * 2
            + tok % 16 // 8) * 4 + d % 4


def value_byte(D, tok, d):
    return ((((((d // 16 * 2 + tok // 32) * 8 + d % 8) * 4 + tok % 8 // 2) * 2 + tok % 32 // 16) * 2
             + d % 16 // 8) * 2 + tok % 16 // 8) * 2 + tok % 2


def byte_order(D, byte):
    """int [64][D]: the byte of each (token, dim)."""
    tok, d = np.meshgrid(np.arange(PAGE), np.arange(D), indexing="ij")
    return byte(D, tok, d)


class Cache:
    """Pages of S sequences; ``pages[s][h]`` is the list of whole pages (codes, scales), ``open[s]`` [2][rows][H][D]."""

    def __init__(self, S, H, D, max_pages):
        self.S, self.H, self.D, self.max_pages = S, H, D, max_pages
        self.pages = [[[] for _ in range(H)] for _ in range(S)]
        self.open = [[np.zeros((0, H, D), np.float32) for _ in range(2)] for _ in range(S)]

    def length(self, s):
        return PAGE * len(self.pages[s][0]) + len(self.open[s][0])

    def append(self, s, k, v):
        """Rows k, v fp32 [n][H][D] of sequence s."""
        rows = [np.concatenate([o, np.asarray(x, np.float32)]) for o, x in zip(self.open[s], (k, v))]
        while len(rows[0]) >= PAGE:
            for h in range(self.H):
                (ck, sk), (cv, sv) = quantize_page(rows[0][:PAGE, h]), quantize_page(rows[1][:PAGE, h])
                self.pages[s][h].append((ck, sk, cv, sv))
            rows = [r[PAGE:] for r in rows]
        self.open[s] = rows

    def held(self, s, h, pages=None):
        """fp64 keys and values [tokens][D] of some whole pages (all by default), then the open rows."""
        take = self.pages[s][h] if pages is None else [self.pages[s][h][p] for p in pages]
        k = [c * np.float64(a) for c, a, _, _ in take] + [self.open[s][0][:, h].astype(np.float64)]
        v = [c * np.float64(a) for _, _, c, a in take] + [self.open[s][1][:, h].astype(np.float64)]
        return np.concatenate(k), np.concatenate(v)


def attention(cache, s, h, q, k_new, v_new, mask, scale, pages=None):
    """One query row q fp64 [D] of KV head h: (out [D], weights of the committed tokens, sum_d |scale q_d k_d| max).

    mask: the new rows it sees."""
    k, v = cache.held(s, h, pages)
    sees = [j for j in range(len(k_new)) if mask >> j & 1]
    k = np.concatenate([k, np.asarray(k_new, np.float64)[sees].reshape(-1, cache.D)])
    v = np.concatenate([v, np.asarray(v_new, np.float64)[sees].reshape(-1, cache.D)])
    if not len(k):
        return np.zeros(cache.D), np.zeros(0), 0.0
    logits = k @ q * scale
    e = np.exp(logits - logits.max())
    w = e / e.sum()
    return w @ v, w[:len(w) - len(sees)], float((np.abs(k) @ np.abs(q)).max() * abs(scale))


def select(cache, s, h, q, top_k, first, last):
    """q fp32 [G][D] -> the ascending list of pages."""
    take = cache.pages[s][h]
    if len(take) <= top_k:
        return list(range(len(take)))
    code, a = quantize_page(q)
    score = []
    for p, (ck, sk, _, _) in enumerate(take):
        best = max(int(ck.sum(axis=0) @ c) for c in code)
        x = np.float32(sk) * np.float32(best)
        score.append(np.inf if np.isnan(x) else x)
    return _best(score, top_k, first, last)


def _best(score, k, first, last):
    """The k best pages, ascending: the first and last ones whatever their score, then by score; equals by the lowest page."""
    n = len(score)
    order = sorted(range(n), key=lambda p: (1, -score[p], p) if first <= p < n - last else (0, 0, p))
    return sorted(order[:k])


def evict(mass, keep, first, last):
    """mass [whole pages] -> (kept pages, dropped pages), both ascending."""
    kept = _best([np.inf if np.isnan(m) else m for m in mass], keep, first, last)
    return kept, sorted(set(range(len(mass))) - set(kept))
