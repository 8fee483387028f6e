"""Key-value cache and attention over it -- oracle, test infrastructure.

The cache is a dict of numpy arrays: ``k`` and ``v`` uint8 codes [pages, Hkv, page, D] with ``ks`` and ``vs`` uint8 E8M0
[pages, Hkv, page, D/32], or uint16 BF16 bits with ``ks`` and ``vs`` None.  ``v`` None is a latent cache.

Pins: hand cases and brute-force loops (tests/test_oracle_attn.py).  The quantiser is oracle/quant.py's with groups of
32 (parity unpinned: no source page fixes a cache's layout).
"""

import numpy as np

from .formats import OCP, bf16_to_f64, e4m3_decode, e8m0_decode
from .quant import group_quant

BLOCK = 32


def write(x_bits, slots, cache, scales):
    """Rows x [T, Hkv, D] (BF16 bits) into a copy of the cache, later rows last: (cache, scales)."""
    cache, scales = cache.copy(), None if scales is None else scales.copy()
    pages, heads, page, D = cache.shape
    for t, slot in enumerate(np.asarray(slots, dtype=np.int64)):
        if not 0 <= slot < pages * page:
            continue
        p, i = divmod(int(slot), page)
        if scales is None:
            cache[p, :, i] = x_bits[t]
        else:
            cache[p, :, i], scales[p, :, i] = group_quant(x_bits[t], BLOCK, OCP)
    return cache, scales


def values(cache, scales):
    """FP64 elements of cache rows [.., D]; a scale of 0xFF makes its block NaN."""
    if scales is None:
        return bf16_to_f64(cache)
    unit = np.repeat(e8m0_decode(scales), BLOCK, axis=-1)
    return e4m3_decode(cache, OCP) * unit


def sequence(cache, scales, table, n):
    """FP64 rows 0..n-1 of one sequence, [n, Hkv, D]; rows whose page is not in the cache are NaN."""
    pages, heads, page, D = cache.shape
    out = np.full((n, heads, D), np.nan)
    for p in range(-(-n // page)):
        rows = min(page, n - p * page)
        if p < len(table) and 0 <= table[p] < pages:
            at = int(table[p])
            out[p * page:p * page + rows] = values(cache[at], None if scales is None else scales[at]).transpose(1, 0, 2)[:rows]
    return out


def attend(q, k, v, scale):
    """Causal attention of the last Lq of Lk tokens: q [Lq, H, D], k and v [Lk, Hkv, D], FP64 -> (out [Lq, H, D], size,
    spread).  size[i,h,:] = sum_j p_j |v_j|, the sum that errors of the weights are relative to; spread[i,h] =
    max_j scale * sum_d |q_d k_jd|, what errors of the scores are relative to.  A row that sees no key is 0."""
    Lq, H, D = q.shape
    Lk, heads = k.shape[:2]
    out, size, spread = np.zeros((Lq, H, D)), np.zeros((Lq, H, D)), np.zeros((Lq, H))
    for h in range(H):
        g = h // (H // heads)
        with np.errstate(invalid="ignore", over="ignore"):
            s = scale * (q[:, h] @ k[:, g].T)
            a = scale * (np.abs(q[:, h]) @ np.abs(k[:, g]).T)
        for i in range(Lq):
            n = min(Lk, Lk - Lq + i + 1)
            if n <= 0:
                continue
            with np.errstate(invalid="ignore", over="ignore"):
                p = np.exp(s[i, :n] - np.max(s[i, :n]))
                p = p / p.sum()
                out[i, h] = p @ v[:n, g]
                size[i, h] = p @ np.abs(v[:n, g])
            spread[i, h] = a[i, :n].max()
    return out, size, spread
