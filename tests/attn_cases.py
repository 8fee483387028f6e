"""Inputs and bounds shared by the tests of the key-value cache and the attention.

Bound of an attention output against the FP64 oracle, from what the kernels round (derived, none fitted):
* the output's own rounding to BF16: 2^-8 |ref|;
* each weight's rounding to BF16 before the second product: 2^-8 of sum p |v| =: size;
* a score's error: the products q_d k_d are exact in FP32, their sum of D terms, the scale and the running maximum's
  subtraction round at most D + 4 times by 2^-24 of spread = scale * sum |q_d k_d|; a weight moves by that much, and the
  sum of weights too: 2 (D + 4) 2^-24 spread size;
* exp2's result 2^-22, and n + 64 roundings of 2^-24 in sums over n keys and their rescaling and joining:
  (n + 128) 2^-24 size.
"""

import numpy as np
import torch

import workloads
from oracle import attn as A
from oracle import formats as F


def bound(ref, size, spread, D, n):
    return 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2 * (D + 4) * 2.0 ** -24 * spread[..., None] + (n + 128) * 2.0 ** -24) * size


def check(got_bits, ref, size, spread, D, n, what=""):
    got = F.bf16_to_f64(got_bits)
    assert got.shape == ref.shape
    assert np.array_equal(np.isnan(got), np.isnan(ref)), what
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), what
    ok = np.isfinite(ref)
    err, lim = np.abs(got - ref)[ok], bound(ref, size, spread, D, n)[ok]
    assert np.all(err <= lim), (what, float((err / np.maximum(lim, 1e-300)).max()), int((err > lim).sum()), err.size)


def normal(rng, *shape):
    return workloads.to_bf16_bits(rng.standard_normal(shape).astype(np.float32))


def make_cache(rng, lens, Hkv, D, page, fp8, latent=False, spare=2):
    """A cache with the pages of len(lens) sequences dealt at random, every page full of finite rows, and its table
    (entries behind a sequence's end are -1)."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    deal = list(rng.permutation(pages))
    table = np.full((len(lens), max(1, max(need, default=1))), -1, np.int32)
    for b, n in enumerate(need):
        table[b, :n] = [deal.pop() for _ in range(n)]
    c = {}
    for name in ("k", "v"):
        if name == "v" and latent:
            c["v"] = c["vs"] = None
        elif fp8:
            x = normal(rng, pages * Hkv * page, D)
            codes, scales = A.group_quant(x, 32, F.OCP)
            c[name] = codes.reshape(pages, Hkv, page, D)
            c[name + "s"] = scales.reshape(pages, Hkv, page, D // 32)
        else:
            c[name], c[name + "s"] = normal(rng, pages, Hkv, page, D), None
    return c, table


def on_gpu(a):
    if a is None:
        return None
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()


def decode_oracle(q_bits, c, table, lens, scale):
    """(out, size, spread) of one new token for each sequence."""
    B, H, D = q_bits.shape
    q = F.bf16_to_f64(q_bits)
    out, size, spread = np.zeros((B, H, D)), np.zeros((B, H, D)), np.zeros((B, H))
    v, vs = (c["k"], c["ks"]) if c["v"] is None else (c["v"], c["vs"])
    for b, n in enumerate(lens):
        if n > 0:
            ks, vv = A.sequence(c["k"], c["ks"], table[b], n), A.sequence(v, vs, table[b], n)
            out[b], size[b], spread[b] = (x[0] for x in A.attend(q[b:b + 1], ks, vv, scale))
    return out, size, spread


def spread_lens(rng, B, total):
    """B lengths of about `total` tokens: two in five empty, one with a third of all, some whole hundreds of 128, the rest at
    random."""
    lens = np.where(rng.random(B) < 0.4, 0, rng.exponential(1.0, B))
    lens = np.floor(lens * total * 2 / 3 / max(lens.sum(), 1e-9)).astype(np.int64)
    lens[::7] = (lens[::7] + 127) // 128 * 128
    lens[B // 2] = total // 3
    return [int(n) for n in lens]


def random_cache(rng, lens, Hkv, D, page, fp8, latent=False):
    """As make_cache, but large: random codes under scales of 2^-9 to 2^-6 (values up to 7, most far smaller), or BF16 of random
    signs and fractions between 2^-3 and 2."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    deal = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), max(need)), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = deal[at:at + n]
        at += n
    c = {"v": None, "vs": None}
    for name in ("k",) if latent else ("k", "v"):
        if fp8:
            x = np.frombuffer(rng.bytes(pages * Hkv * page * D), np.uint8).reshape(pages, Hkv, page, D).copy()
            x[(x & 0x7F) == 0x7F] = 0
            c[name], c[name + "s"] = x, rng.integers(118, 122, (pages, Hkv, page, D // 32)).astype(np.uint8)
        else:
            x = np.frombuffer(rng.bytes(pages * Hkv * page * D * 2), np.uint16).reshape(pages, Hkv, page, D)
            c[name], c[name + "s"] = (x & 0x81FF) + 0x3E00, None
    return c, table


def sampled_oracle(q_bits, c, table, lens, scale, heads):
    """decode_oracle for some of the heads, in FP64 without a loop over rows."""
    B, H, D = q_bits.shape
    Hkv = c["k"].shape[1]
    q = F.bf16_to_f64(q_bits[:, heads])
    out, size, spread = np.zeros((B, len(heads), D)), np.zeros((B, len(heads), D)), np.zeros((B, len(heads)))
    for b, n in enumerate(lens):
        for g in sorted({h // (H // Hkv) for h in heads}) if n > 0 else ():
            rows = [A.sequence(c[x][:, g:g + 1], None if c[x + "s"] is None else c[x + "s"][:, g:g + 1], table[b], n)[:, 0]
                    for x in (("k",) if c["v"] is None else ("k", "v"))]
            k, v = rows[0], rows[-1]
            mine = [i for i, h in enumerate(heads) if h // (H // Hkv) == g]
            s = scale * (q[b, mine] @ k.T)
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            out[b, mine], size[b, mine] = p @ v, p @ np.abs(v)
            spread[b, mine] = scale * (np.abs(q[b, mine]) @ np.abs(k).T).max(1)
    return out, size, spread
