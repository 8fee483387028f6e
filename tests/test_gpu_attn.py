"""The key-value cache and the attention over it on the GPU against the FP64 oracle (bounds: attn_cases.py; the cache's
bytes and the rows read back are equal)."""

import numpy as np
import pytest
import torch

import mx_scaled_fp8_amd as mx
import workloads
from attn_cases import check, decode_oracle, make_cache, normal, on_gpu
from helpers import dev_i64, host_u16, host_u8, requires_gpu, say
from oracle import attn as A
from oracle import formats as F

pytestmark = [pytest.mark.gpu, requires_gpu, pytest.mark.timeout(300)]

KINDS = pytest.mark.parametrize("fp8", [True, False], ids=["mxfp8", "bf16"])


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


# ------------------------------------------------------------------- write

def _empty(rng, pages, Hkv, page, D, fp8):
    if fp8:
        return rng.integers(0, 256, (pages, Hkv, page, D)).astype(np.uint8), rng.integers(0, 256, (pages, Hkv, page, D // 32)).astype(np.uint8)
    return rng.integers(0, 65536, (pages, Hkv, page, D)).astype(np.uint16), None


def _same(dev, host):
    if host is not None:
        assert np.array_equal(host_u16(dev) if host.dtype == np.uint16 else host_u8(dev), host)


@pytest.mark.parametrize("T,Hkv,D,page", [(1, 1, 32, 16), (1, 8, 128, 64), (7, 3, 64, 16), (65, 2, 96, 128), (130, 1, 512, 64),
                                          (33, 5, 1024, 32), (1000, 8, 128, 4096)])
@KINDS
@pytest.mark.parametrize("latent", [False, True])
def test_write(T, Hkv, D, page, fp8, latent):
    """Rows out of a fused projection, some slots outside the cache; every byte that no row owns stays."""
    rng = np.random.default_rng(T + D + page)
    pages = -(-T // page) + 2
    x = workloads.activations(rng, T, 3 * Hkv * D).reshape(T, 3 * Hkv, D)
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    slots[T // 2::5] = rng.choice([-1, -7, pages * page, 1 << 40], slots[T // 2::5].shape)
    kc, ks = _empty(rng, pages, Hkv, page, D, fp8)
    vc, vs = (None, None) if latent else _empty(rng, pages, Hkv, page, D, fp8)
    dx = on_gpu(x)
    dk, dks, dv, dvs = (on_gpu(a) for a in (kc, ks, vc, vs))
    say("kv write", T, Hkv, D, page, fp8, latent)
    mx.mx_kv_cache_write(dx[:, Hkv:2 * Hkv], None if latent else dx[:, 2 * Hkv:], dev_i64(slots), dk, dv, k_scale=dks, v_scale=dvs)
    torch.cuda.synchronize()
    rk, rks = A.write(x[:, Hkv:2 * Hkv], slots, kc, ks)
    _same(dk, rk)
    _same(dks, rks)
    if not latent:
        rv, rvs = A.write(x[:, 2 * Hkv:], slots, vc, vs)
        _same(dv, rv)
        _same(dvs, rvs)


def test_write_blocks_of_zeros_infinities_nan_and_the_smallest():
    rows = np.zeros((8, 1, 64), np.uint16)
    rows[1, 0, 40] = 0x7F80                        # Inf in the second block
    rows[2, 0, 0] = 0xFF80
    rows[3, 0, 63] = 0x7FC1                        # NaN
    rows[4] = 0x0001                               # the smallest subnormal
    rows[5] = 0x7F7F                               # the largest
    rows[6, 0, :32], rows[6, 0, 32:] = 0x8000, 0xBF80
    rows[7, 0, ::2] = 0x43E0                       # 448
    kc, ks = np.full((1, 1, 16, 64), 0xAA, np.uint8), np.full((1, 1, 16, 2), 0xAA, np.uint8)
    dk, dks = on_gpu(kc), on_gpu(ks)
    slots = np.arange(8) * 2
    say("kv write special")
    mx.mx_kv_cache_write(on_gpu(rows), None, dev_i64(slots), dk, None, k_scale=dks)
    torch.cuda.synchronize()
    rk, rks = A.write(rows, slots, kc, ks)
    _same(dk, rk)
    _same(dks, rks)


# -------------------------------------------------------------------- read

@pytest.mark.parametrize("lens,Hkv,D,page", [([1], 1, 32, 16), ([5, 0, 17, 1], 2, 96, 16), ([130, 64, 63, 65], 8, 128, 64),
                                             ([0, 0, 33], 3, 64, 32), ([700], 1, 512, 4096), ([1] * 70, 1, 64, 16)])
@KINDS
@pytest.mark.parametrize("latent", [False, True])
def test_read(lens, Hkv, D, page, fp8, latent):
    rng = np.random.default_rng(sum(lens) + D)
    c, table = make_cache(rng, lens, Hkv, D, page, fp8, latent)
    before, behind = 3, 5                            # rows that no sequence owns
    offsets = before + np.concatenate([[0], np.cumsum(lens)])
    rows = int(offsets[-1]) + behind
    mark = np.full((rows, Hkv, D), 0x1234, np.uint16)
    k, v = on_gpu(mark), None if latent else on_gpu(mark)
    say("kv read", lens[:4], Hkv, D, page, fp8, latent)
    mx.mx_kv_cache_read(on_gpu(c["k"]), on_gpu(c["v"]), _i32(table), _i32(offsets), rows, k_scale=on_gpu(c["ks"]),
                        v_scale=on_gpu(c["vs"]), k=k, v=v)
    torch.cuda.synchronize()
    for name, got in (("k", k), ("v", v)):
        if got is not None:
            want = mark.copy()
            for b, n in enumerate(lens):
                want[offsets[b]:offsets[b + 1]] = F.f64_to_bf16_rne(A.sequence(c[name], c[name + "s"], table[b], n))
            assert np.array_equal(host_u16(got), want)


@KINDS
def test_read_bad_pages_and_nan_scales(fp8):
    """Pages outside the cache and tokens behind the table are NaN and read nothing; a scale of 0xFF makes its block NaN
    whatever the codes are."""
    rng = np.random.default_rng(3)
    c, table = make_cache(rng, [40, 40, 16], 2, 64, 16, fp8)
    table[0, 1], table[1, 2] = -1, 1 << 30
    if fp8:
        c["ks"][table[2, 0], 1, 5, 0] = 0xFF
        c["ks"][table[2, 0], 0, 6, 1] = 0
    lens = [40, 48, 16]                              # the second is longer than its pages are good for
    offsets = np.concatenate([[0], np.cumsum(lens)])
    say("kv read bad pages", fp8)
    k, v = mx.mx_kv_cache_read(on_gpu(c["k"]), on_gpu(c["v"]), _i32(table), _i32(offsets), int(offsets[-1]),
                               k_scale=on_gpu(c["ks"]), v_scale=on_gpu(c["vs"]))
    torch.cuda.synchronize()
    for name, got in (("k", k), ("v", v)):
        want = np.concatenate([A.sequence(c[name], c[name + "s"], table[b], n) for b, n in enumerate(lens)])
        g = F.bf16_to_f64(host_u16(got))
        assert np.array_equal(np.isnan(g), np.isnan(want))
        assert np.array_equal(g[~np.isnan(g)], F.bf16_to_f64(F.f64_to_bf16_rne(want[~np.isnan(want)])))


# ------------------------------------------------------------------ decode

def _decode(rng, lens, Hkv, G, D, page, fp8, latent=False, scale=None):
    c, table = make_cache(rng, lens, Hkv, D, page, fp8, latent)
    q = normal(rng, len(lens), Hkv * G, D)
    say("decode", lens[:4], Hkv, G, D, page, fp8, latent)
    out = mx.mx_attn_decode(on_gpu(q), on_gpu(c["k"]), on_gpu(c["v"]), _i32(table), _i32(lens), k_scale=on_gpu(c["ks"]),
                            v_scale=on_gpu(c["vs"]), scale=scale)
    torch.cuda.synchronize()
    ref = decode_oracle(q, c, table, lens, D ** -0.5 if scale is None else scale)
    check(host_u16(out), *ref, D, max(lens), "decode")


@pytest.mark.parametrize("lens,Hkv,G,page", [([1], 1, 1, 16), ([15, 16, 17], 2, 4, 16), ([31, 32, 33, 0, 127, 128, 129], 1, 8, 32),
                                             ([0], 2, 2, 16), ([1000, 3, 512], 2, 16, 64), ([257, 1], 1, 17, 16),
                                             ([300], 1, 40, 128), ([2000, 1500], 3, 5, 1024)])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
@KINDS
def test_decode(lens, Hkv, G, page, D, fp8):
    _decode(np.random.default_rng(sum(lens) + G + D), lens, Hkv, G, D, page, fp8)


@pytest.mark.parametrize("lens,G,D,page", [([700, 33, 129], 128, 512, 64), ([64], 16, 512, 16), ([90, 1], 3, 128, 16), ([0, 31, 32, 65], 32, 512, 16),
                                           ([1500, 0, 2], 130, 512, 128), ([200], 33, 64, 32), ([64, 63, 1], 100, 256, 16), ([300, 5], 64, 128, 16)])
@KINDS
def test_decode_latent(lens, G, D, page, fp8):
    _decode(np.random.default_rng(G), lens, 1, G, D, page, fp8, latent=True, scale=0.11)


@pytest.mark.parametrize("lens,Hkv,G,D", [([130, 63, 0, 64], 2, 32, 64), ([257, 7], 1, 71, 128), ([33, 500], 1, 128, 256), ([70], 2, 40, 512)])
@KINDS
def test_decode_many_heads_a_key_head(lens, Hkv, G, D, fp8):
    _decode(np.random.default_rng(G), lens, Hkv, G, D, 32, fp8)


@pytest.mark.parametrize("B", [300, 1030])
def test_decode_many_sequences(B):
    """More sequences than threads, many empty."""
    rng = np.random.default_rng(B)
    lens = [int(n) if n > 0 else 0 for n in rng.integers(-40, 150, B)]
    _decode(rng, lens, 1, 2, 64, 32, True)
    _decode(rng, lens, 1, 2, 64, 32, False)


# ----------------------------------------------------------------- prefill

def _prefill(rng, lens, past, Hkv, G, D, same=False, scale=None):
    """lens rows of q over past + lens keys each; past may be negative (rows without keys)."""
    H = Hkv * G
    keys = [max(0, n + p) for n, p in zip(lens, past)]
    qo, ko = np.concatenate([[0], np.cumsum(lens)]), np.concatenate([[0], np.cumsum(keys)])
    q, k = normal(rng, qo[-1], H, D), normal(rng, ko[-1], Hkv, D)
    v = k if same else normal(rng, ko[-1], Hkv, D)
    dk = on_gpu(k)
    say("prefill", lens[:4], past[:4], Hkv, G, D, same)
    out = mx.mx_attn_prefill(on_gpu(q), dk, dk if same else on_gpu(v), _i32(qo), _i32(ko), scale=scale)
    torch.cuda.synchronize()
    sc = D ** -0.5 if scale is None else scale
    f = F.bf16_to_f64
    parts = [A.attend(f(q[qo[b]:qo[b + 1]]), f(k[ko[b]:ko[b + 1]]), f(v[ko[b]:ko[b + 1]]), sc) for b in range(len(lens))]
    check(host_u16(out), *(np.concatenate([p[i] for p in parts]) for i in range(3)), D, max(keys + [1]), "prefill")


@pytest.mark.parametrize("lens,past,Hkv,G", [([1], [0], 1, 1), ([31, 32, 33], [0, 0, 0], 2, 1), ([127, 128, 129, 1], [0] * 4, 1, 3),
                                             ([5, 0, 70], [0, 0, 0], 1, 2), ([1, 7, 130], [63, 64, 500], 2, 2),
                                             ([300], [0], 1, 4), ([40, 20], [-10, -20], 1, 2), ([64], [1000], 1, 1)])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_prefill(lens, past, Hkv, G, D):
    _prefill(np.random.default_rng(sum(lens) + D), lens, past, Hkv, G, D)


@pytest.mark.parametrize("D", [128, 512])
def test_prefill_latent(D):
    _prefill(np.random.default_rng(D), [90, 200], [0, 33], 1, 16, D, same=True, scale=0.07)
