"""The key-value cache and the attention over it on the GPU against the FP64 oracle (bounds: attn_cases.py; the cache's
bytes and the rows read back are equal)."""

import numpy as np
import pytest
import torch

import mx_scaled_fp8_amd as mx
import workloads
from attn_cases import check, decode_oracle, make_cache, normal, on_gpu, random_cache, sampled_oracle, spread_lens
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


# ------------------------------------------- values that hide, and do not

def _poison_behind(c, table, lens, fp8):
    """NaN, Inf and the largest values in every cache row that no sequence owns."""
    pages, Hkv, page, D = c["k"].shape
    owned = np.zeros((pages, page), bool)
    for b, n in enumerate(lens):
        for i in range(n):
            owned[table[b, i // page], i % page] = True
    where = np.broadcast_to(~owned[:, None, :], (pages, Hkv, page))
    for name in ("k", "v"):
        if c[name] is None:
            continue
        if fp8:
            c[name][where] = 0x7F
            c[name + "s"][where] = 0xFF
        else:
            c[name][where] = np.resize(np.array([0x7FC0, 0x7F80, 0xFF80, 0x7F7F], np.uint16), D)


@pytest.mark.parametrize("Hkv,G,D,page,latent", [(2, 4, 128, 16, False), (2, 3, 64, 64, False), (1, 5, 512, 16, False), (1, 2, 256, 32, True),
                                                 (1, 64, 512, 64, True), (1, 40, 128, 16, False), (1, 33, 256, 64, True), (2, 32, 64, 16, False)])
@KINDS
def test_decode_ignores_what_lies_behind_the_end(Hkv, G, D, page, latent, fp8):
    rng = np.random.default_rng(G)
    lens = [1, 15, 33, 70, 0, 129, 600]
    c, table = make_cache(rng, lens, Hkv, D, page, fp8, latent)
    _poison_behind(c, table, lens, fp8)
    q = normal(rng, len(lens), Hkv * G, D)
    say("decode behind the end", Hkv, G, D, page, latent, fp8)
    out = mx.mx_attn_decode(on_gpu(q), on_gpu(c["k"]), on_gpu(c["v"]), _i32(table), _i32(lens), k_scale=on_gpu(c["ks"]),
                            v_scale=on_gpu(c["vs"]))
    torch.cuda.synchronize()
    check(host_u16(out), *decode_oracle(q, c, table, lens, D ** -0.5), D, max(lens))


@pytest.mark.parametrize("Hkv,G,D,latent", [(2, 4, 128, False), (1, 64, 512, True), (1, 40, 128, False), (1, 3, 512, False)])
@KINDS
def test_decode_bad_pages_and_lengths(Hkv, G, D, latent, fp8):
    """A sequence with a page outside the cache or longer than its table has NaN outputs, its neighbours are untouched."""
    rng = np.random.default_rng(G)
    lens = [700, 300, 90, 40, 512]
    c, table = make_cache(rng, lens, Hkv, D, 32, fp8, latent)
    q = normal(rng, len(lens), Hkv * G, D)
    table[1, 5], table[3, 1] = c["k"].shape[0], -3
    say("decode bad pages", Hkv, G, D, latent, fp8)
    asked = [700, 300, 90, 40, table.shape[1] * 32 + 1]
    out = mx.mx_attn_decode(on_gpu(q), on_gpu(c["k"]), on_gpu(c["v"]), _i32(table), _i32(asked), k_scale=on_gpu(c["ks"]),
                            v_scale=on_gpu(c["vs"]))
    torch.cuda.synchronize()
    got = host_u16(out)
    assert np.isnan(F.bf16_to_f64(got[[1, 3, 4]])).all()
    ref = [x[[0, 2]] for x in decode_oracle(q, c, table, lens, D ** -0.5)]
    check(got[[0, 2]], *ref, D, 700)


@pytest.mark.parametrize("G,D,latent", [(4, 128, False), (64, 512, True), (2, 512, False)])
@KINDS
def test_decode_values_that_are_not_finite_count(G, D, latent, fp8):
    """A NaN or Inf that a sequence does see reaches its outputs, and no other sequence's."""
    rng = np.random.default_rng(G)
    lens = [100, 100, 40]
    c, table = make_cache(rng, lens, 1, D, 16, fp8, latent)
    name = "k" if latent else "v"
    if fp8:
        c[name + "s"][table[1, 2], 0, 3, 1] = 0xFF                  # token 35, elements 32..63
    else:
        c[name][table[1, 2], 0, 3, 40] = 0x7F80 if not latent else 0x7FC0
    q = normal(rng, 3, G, D)
    say("decode not finite", G, D, latent, fp8)
    out = mx.mx_attn_decode(on_gpu(q), on_gpu(c["k"]), on_gpu(c["v"]), _i32(table), _i32(lens), k_scale=on_gpu(c["ks"]),
                            v_scale=on_gpu(c["vs"]))
    torch.cuda.synchronize()
    ref = decode_oracle(q, c, table, lens, D ** -0.5)
    assert not np.isfinite(ref[0][1]).all() and np.isfinite(ref[0][[0, 2]]).all()
    check(host_u16(out), *ref, D, 100)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("same", [False, True])
@pytest.mark.parametrize("G", [1, 4])
def test_prefill_keys_and_values_that_a_row_does_not_see(D, same, G):
    """NaN and infinities in keys and values reach the rows that see them, each as itself, and no other row."""
    rng = np.random.default_rng(D + G)
    Lq = 150
    q, k = normal(rng, Lq, G, D), normal(rng, Lq, 1, D)
    v = k if same else normal(rng, Lq, 1, D)
    v[140, 0, 3] = 0x7FC0
    if not same:
        v[60, 0, :40] = 0x7F80                       # +Inf
        v[61, 0, 5] = 0xFF80                         # -Inf, seen from row 61 on: with +Inf, NaN
        v[97, 0, D - 1] = 0xFF80
        k[120] = 0x7F80                              # scores of +-Inf or NaN
    say("prefill not finite", D, same, G)
    dk = on_gpu(k)
    out = mx.mx_attn_prefill(on_gpu(q), dk, dk if same else on_gpu(v), _i32([0, Lq]), _i32([0, Lq]))
    torch.cuda.synchronize()
    f = F.bf16_to_f64
    ref = A.attend(f(q), f(k), f(v), D ** -0.5)
    assert np.isfinite(ref[0][:60]).all() and np.isnan(ref[0][140:]).any()
    check(host_u16(out), *ref, D, Lq)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_prefill_scores_that_grow(D):
    """Maxima that move in steps above and below what lets the weights stand, and scores far apart."""
    Lk = 400
    q = np.zeros((Lk, 1, D), np.float32)
    k = np.zeros((Lk, 1, D), np.float32)
    q[:, 0, 0] = 1
    steps = np.concatenate([np.arange(100) * 0.9, 90 + np.arange(100) * 7.0, 790 - np.arange(100) * 11.0, np.full(100, -300.0)])
    k[:, 0, 0] = steps
    v = np.random.default_rng(D).standard_normal((Lk, 1, D)).astype(np.float32)
    q, k, v = (workloads.to_bf16_bits(x) for x in (q, k, v))
    say("prefill growing scores", D)
    out = mx.mx_attn_prefill(on_gpu(q), on_gpu(k), on_gpu(v), _i32([0, Lk]), _i32([0, Lk]), scale=1.0)
    c = {"k": k.reshape(25, 1, 16, D), "v": v.reshape(25, 1, 16, D), "ks": None, "vs": None}
    table = np.arange(25, dtype=np.int32)[None]
    dec = mx.mx_attn_decode(on_gpu(q[:1]), on_gpu(c["k"]), on_gpu(c["v"]), _i32(table), _i32([Lk]), scale=1.0)
    torch.cuda.synchronize()
    f = F.bf16_to_f64
    ref = A.attend(f(q), f(k), f(v), 1.0)
    check(host_u16(out), *ref, D, Lk)
    check(host_u16(dec), *decode_oracle(q[:1], c, table, [Lk], 1.0), D, Lk)


# ------------------------------------ strides, rows left alone, repetition

@pytest.mark.parametrize("D", [64, 512])
def test_strided_rows_and_rows_that_no_prompt_owns(D):
    """q, k and v as slices of one fused projection; rows before the first and behind the last prompt stay as they were."""
    rng = np.random.default_rng(D)
    H, Hkv, before, lens, behind = 4, 2, 5, [33, 0, 140], 9
    T = before + sum(lens) + behind
    fused = normal(rng, T, H + 2 * Hkv + 1, D)
    offsets = before + np.concatenate([[0], np.cumsum(lens)])
    d = on_gpu(fused)
    out = on_gpu(np.full((T, H, D), 0x1234, np.uint16))
    say("prefill strided", D)
    mx.mx_attn_prefill(d[:, :H], d[:, H:H + Hkv], d[:, H + Hkv:H + 2 * Hkv], _i32(offsets), _i32(offsets), out=out)
    torch.cuda.synchronize()
    got, f = host_u16(out), F.bf16_to_f64(fused)
    assert np.all(got[:before] == 0x1234) and np.all(got[T - behind:] == 0x1234)
    for b in range(len(lens)):
        x = slice(offsets[b], offsets[b + 1])
        if lens[b]:
            check(got[x], *A.attend(f[x, :H], f[x, H:H + Hkv], f[x, H + Hkv:H + 2 * Hkv], D ** -0.5), D, lens[b])


@KINDS
def test_decode_strided_queries_and_given_output(fp8):
    rng = np.random.default_rng(1)
    lens, Hkv, G, D = [200, 3], 2, 4, 128
    c, table = make_cache(rng, lens, Hkv, D, 16, fp8)
    fused = normal(rng, 2, 3 * Hkv * G, D)
    out = torch.zeros((2, Hkv * G * D), dtype=torch.bfloat16, device="cuda")
    ws = torch.full((mx.mx_attn_decode_workspace_bytes(2, Hkv * G, Hkv, D, table.shape[1], 16),), 0xFF, dtype=torch.uint8, device="cuda")
    say("decode strided", fp8)
    got = mx.mx_attn_decode(on_gpu(fused)[:, 4:4 + Hkv * G], on_gpu(c["k"]), on_gpu(c["v"]), _i32(table), _i32(lens),
                            k_scale=on_gpu(c["ks"]), v_scale=on_gpu(c["vs"]), out=out, workspace=ws)
    torch.cuda.synchronize()
    assert got is out
    ref = decode_oracle(fused[:, 4:4 + Hkv * G], c, table, lens, D ** -0.5)
    check(host_u16(out).reshape(2, Hkv * G, D), *ref, D, 200)


def _chain(rng, fp8):
    lens, Hkv, G, D = [900, 1500, 64], 2, 8, 128
    c, table = make_cache(rng, lens, Hkv, D, 64, fp8)
    q = on_gpu(normal(rng, 3, Hkv * G, D)).view(torch.bfloat16)
    return [q] + [on_gpu(c[n]) for n in ("k", "v", "ks", "vs")] + [_i32(table), _i32(lens)]


@KINDS
def test_repetition_other_streams_and_stale_workspaces(fp8):
    """The same call gives the same bits whatever the workspace held, on any stream, two at once."""
    q, k, v, ks, vs, table, lens = _chain(np.random.default_rng(2), fp8)
    call = lambda **kw: mx.mx_attn_decode(q, k, v, table, lens, k_scale=ks, v_scale=vs, **kw)  # noqa: E731
    need = mx.mx_attn_decode_workspace_bytes(3, 16, 2, 128, table.shape[1], 64)
    say("decode repeated", fp8)
    first = call()
    dirty = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            outs += [call(workspace=dirty.clone()) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(first.view(torch.int16), o.view(torch.int16)) for o in outs)
    rows = 700
    x = on_gpu(normal(np.random.default_rng(3), rows, 16, 128))
    kk = on_gpu(normal(np.random.default_rng(4), 9000, 2, 128))
    qo, ko = _i32([0, rows]), _i32([0, 9000])
    a = mx.mx_attn_prefill(x, kk, kk.clone(), qo, ko)
    w = torch.full((max(1, mx.mx_attn_prefill_workspace_bytes(1, rows, 9000, 16, 2, 128)),), 0xFF, dtype=torch.uint8, device="cuda")
    b = mx.mx_attn_prefill(x, kk, kk.clone(), qo, ko, workspace=w)
    torch.cuda.synchronize()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@KINDS
def test_graph_step_by_step(fp8):
    """A decode step (write the new token, attend) and a prompt captured once and replayed with other contents: every
    replay equals the eager calls."""
    rng = np.random.default_rng(5)
    B, Hkv, G, D, page = 3, 2, 4, 128, 16
    c, table = make_cache(rng, [200] * B, Hkv, D, page, fp8)
    k, v, ks, vs = (on_gpu(c[n]) for n in ("k", "v", "ks", "vs"))
    table_d, lens, slots = _i32(table), _i32([5, 60, 130]), dev_i64([0] * B)
    rows = on_gpu(normal(rng, B, (G + 2) * Hkv, D))
    prompt = on_gpu(normal(rng, 90, Hkv * G, D))
    keys = on_gpu(normal(rng, 4000, Hkv, D))
    qo, ko = _i32([0, 30, 90]), _i32([0, 3000, 4000])

    def step():
        mx.mx_kv_cache_write(rows[:, G * Hkv:(G + 1) * Hkv], rows[:, (G + 1) * Hkv:], slots, k, v, k_scale=ks, v_scale=vs)
        return (mx.mx_attn_decode(rows[:, :G * Hkv], k, v, table_d, lens, k_scale=ks, v_scale=vs),
                mx.mx_attn_prefill(prompt, keys, keys, qo, ko))

    say("graph", fp8)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step()
    for n in range(4):
        at = [5 + n, 60 + 3 * n, 130 + n]
        lens.copy_(_i32([x + 1 for x in at]))
        slots.copy_(dev_i64([int(table[b, at[b] // page]) * page + at[b] % page for b in range(B)]))
        rows.copy_(on_gpu(normal(rng, B, (G + 2) * Hkv, D)))
        prompt.copy_(on_gpu(normal(rng, 90, Hkv * G, D)))
        ko.copy_(_i32([0, 2000 + 17 * n, 4000 - n]))
        g.replay()
        torch.cuda.synchronize()
        got = [h.clone() for h in held]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(got, want)), n


# ------------------------------------------------------------- used together

def test_prompt_in_chunks_then_tokens_then_the_output_projection():
    """A prompt in two chunks through an MXFP8 cache: write, read back, attend; then new tokens; then the inverse rotation
    and quantisation of the output projection.  Each step against the oracle on what the cache then holds."""
    rng = np.random.default_rng(6)
    H, Hkv, D, page, first, second = 8, 2, 128, 16, 70, 50
    n = first + second
    pages = 12
    k, v = (torch.zeros((pages, Hkv, page, D), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((pages, Hkv, page, D // 32), dtype=torch.uint8, device="cuda") for _ in range(2))
    table = rng.permutation(pages)[None, :9].astype(np.int32)
    slot = lambda i: int(table[0, i // page]) * page + i % page  # noqa: E731
    f = F.bf16_to_f64
    host = lambda: {"k": host_u8(k), "v": host_u8(v), "ks": host_u8(ks), "vs": host_u8(vs)}  # noqa: E731
    say("chunks")
    for begin, end in ((0, first), (first, n)):
        rows = normal(rng, end - begin, H + 2 * Hkv, D)
        d = on_gpu(rows)
        mx.mx_kv_cache_write(d[:, H:H + Hkv], d[:, H + Hkv:], dev_i64([slot(i) for i in range(begin, end)]), k, v, k_scale=ks, v_scale=vs)
        kk, vv = mx.mx_kv_cache_read(k, v, _i32(table), _i32([0, end]), end, k_scale=ks, v_scale=vs)
        out = mx.mx_attn_prefill(d[:, :H], kk, vv, _i32([0, end - begin]), _i32([0, end]))
        torch.cuda.synchronize()
        c = host()
        ref = A.attend(f(rows[:, :H]), A.sequence(c["k"], c["ks"], table[0], end), A.sequence(c["v"], c["vs"], table[0], end), D ** -0.5)
        check(host_u16(out), *ref, D, end, "chunk")
    for i in range(n, n + 3):
        rows = normal(rng, 1, H + 2 * Hkv, D)
        d = on_gpu(rows)
        mx.mx_kv_cache_write(d[:, H:H + Hkv], d[:, H + Hkv:], dev_i64([slot(i)]), k, v, k_scale=ks, v_scale=vs)
        out = mx.mx_attn_decode(d[:, :H], k, v, _i32(table), _i32([i + 1]), k_scale=ks, v_scale=vs)
        torch.cuda.synchronize()
        check(host_u16(out), *decode_oracle(rows[:, :H], host(), table, [i + 1], D ** -0.5), D, i + 1, "token")
    cos, sin = workloads.rope_tables(rows=256)
    q, s = mx.mx_inv_rope_group_quant(out.view(1, H * D), dev_i64([n + 2]), on_gpu(cos), on_gpu(sin), H, D, 64)
    torch.cuda.synchronize()
    from oracle.quant import inv_rope_group_quant
    rq, rs = inv_rope_group_quant(host_u16(out).reshape(1, H * D), np.array([n + 2]), cos, sin, H, D, 64)
    assert np.array_equal(host_u8(s), rs) and (host_u8(q) != rq).sum() <= 1


# ------------------------------------------------------- behind 32-bit offsets

@KINDS
def test_pages_behind_4_gb(fp8):
    """A cache of more than 2^32 bytes whose sequences are in its last pages (and its first)."""
    rng = np.random.default_rng(7)
    Hkv, G, D, page = 8, 2, 128, 64
    per_page = Hkv * page * D * (1 if fp8 else 2)
    pages = (9 << 30) // 2 // per_page
    dtype = torch.uint8 if fp8 else torch.bfloat16
    k = torch.empty((pages, Hkv, page, D), dtype=dtype, device="cuda")
    v = torch.empty((pages, Hkv, page, D), dtype=dtype, device="cuda")
    ks, vs = (torch.empty((pages, Hkv, page, D // 32), dtype=torch.uint8, device="cuda") if fp8 else None for _ in range(2))
    lens = [100, 300]
    table = np.array([[pages - 1, 0, 0, 0, 0], [pages - 2, 1, pages - 7, pages // 2, pages - 3]], np.int32)
    rows = normal(rng, sum(lens), (2 + G) * Hkv, D)
    d = on_gpu(rows).view(torch.bfloat16)
    slots = [int(table[b, i // page]) * page + i % page for b, n in enumerate(lens) for i in range(n)]
    say("behind 4 GB", fp8)
    mx.mx_kv_cache_write(d[:, :Hkv], d[:, Hkv:2 * Hkv], dev_i64(slots), k, v, k_scale=ks, v_scale=vs)
    q = d[:2, 2 * Hkv:]
    out = mx.mx_attn_decode(q, k, v, _i32(table), _i32(lens), k_scale=ks, v_scale=vs)
    offsets = [0, 100, 400]
    kk, vv = mx.mx_kv_cache_read(k, v, _i32(table), _i32(offsets), 400, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    kh, vh = F.bf16_to_f64(host_u16(kk)), F.bf16_to_f64(host_u16(vv))
    if not fp8:
        assert np.array_equal(host_u16(kk), rows[:, :Hkv]) and np.array_equal(host_u16(vv), rows[:, Hkv:2 * Hkv])
    else:
        codes, sc = A.group_quant(rows[:, :Hkv].reshape(-1, D), 32, F.OCP)
        assert np.array_equal(kh, A.values(codes, sc).reshape(400, Hkv, D))
    qh = F.bf16_to_f64(rows[:2, 2 * Hkv:])
    parts = [A.attend(qh[b:b + 1], kh[offsets[b]:offsets[b + 1]], vh[offsets[b]:offsets[b + 1]], D ** -0.5) for b in range(2)]
    check(host_u16(out), *(np.concatenate([p[i] for p in parts]) for i in range(3)), D, 300)


def test_prompt_rows_behind_4_gb():
    """q, k, v and out rows whose offsets pass 2^32 bytes."""
    rng = np.random.default_rng(8)
    D, Hkv, H, T = 128, 2, 4, 600000
    k = torch.zeros((T, 16, Hkv, D), dtype=torch.bfloat16, device="cuda")[:, 3]       # rows 8 KiB apart
    q = torch.zeros((T, 8, H, D), dtype=torch.bfloat16, device="cuda")[:, 5]
    n = 200
    rows, keys = normal(rng, n, H, D), normal(rng, n, Hkv, D)
    q[T - n:], k[T - n:] = on_gpu(rows).view(torch.bfloat16), on_gpu(keys).view(torch.bfloat16)
    offsets = _i32([T - n, T])
    say("prompt behind 4 GB")
    out = mx.mx_attn_prefill(q, k, k, offsets, offsets)
    torch.cuda.synchronize()
    f = F.bf16_to_f64
    check(host_u16(out[T - n:]), *A.attend(f(rows), f(keys), f(keys), D ** -0.5), D, n)


# ------------------------------------------------- refusals of the binding

def _z(*shape, dtype=torch.uint8):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def _raises(match, f, *a, **kw):
    with pytest.raises((ValueError, TypeError, mx.MxError), match=match):
        f(*a, **kw)


def test_binding_refusals():
    bf, i32, i64 = torch.bfloat16, torch.int32, torch.int64
    kc, sc, kb = _z(4, 2, 16, 64), _z(4, 2, 16, 2), _z(4, 2, 16, 64, dtype=bf)
    rows, slots, table, lens = _z(3, 2, 64, dtype=bf), _z(3, dtype=i64), _z(3, 2, dtype=i32), _z(3, dtype=i32)
    say("refusals")
    w = mx.mx_kv_cache_write
    _raises("k must be", w, _z(6, 64, dtype=bf), rows, slots, kc, kc, sc, sc)
    _raises("k has shape", w, _z(3, 1, 64, dtype=bf), rows, slots, kc, kc, sc, sc)
    _raises("k must be", w, rows.float(), rows, slots, kc, kc, sc, sc)
    _raises("dense heads", w, _z(3, 64, 2, dtype=bf).transpose(1, 2), rows, slots, kc, kc, sc, sc)
    _raises("v has shape", w, rows, rows[:2], slots, kc, kc, sc, sc)
    _raises("go together", w, rows, None, slots, kc, kc.clone(), sc, sc.clone())
    _raises("slots has", w, rows, rows, slots[:2], kc, kc, sc, sc)
    _raises("slots must be", w, rows, rows, slots.int(), kc, kc, sc, sc)
    _raises("k_cache must be", w, rows, rows, slots, kc[0], kc, sc, sc)
    _raises("v_cache has shape", w, rows, rows, slots, kc, kc[:3], sc, sc)
    _raises("k_scale", w, rows, rows, slots, kc, kc, None, sc)
    _raises("v_scale", w, rows, rows, slots, kc, kc, sc, None)
    _raises("k_scale", w, rows, rows, slots, kb, kb, sc, sc)
    _raises("k_scale has shape", w, rows, rows, slots, kc, kc, _z(4, 2, 16, 4), sc)
    _raises("contiguous", w, rows, rows, slots, _z(4, 2, 16, 128)[..., :64], kc, sc, sc)
    _raises("overlaps", w, rows, rows, slots, kc, kc, sc, sc.clone())
    r = mx.mx_kv_cache_read
    _raises("block_table must be", r, kb, kb, table[0], lens, 3)
    _raises("block_table must be", r, kb, kb, table.long(), lens, 3)
    _raises("offsets has", r, kb, kb, table, lens, 3)
    _raises("negative", r, kb, kb, table, _z(4, dtype=i32), -1)
    _raises("k has", r, kb, kb, table, _z(4, dtype=i32), 3, k=rows[:2])
    _raises("v must be None", r, kb, None, table, _z(4, dtype=i32), 3, v=rows)
    d = mx.mx_attn_decode
    q = _z(3, 4, 64, dtype=bf)
    _raises("q has 2 rows", d, q[:2], kb, kb, table, lens)
    _raises("q has shape", d, _z(3, 4, 128, dtype=bf), kb, kb, table, lens)
    _raises("lens has", d, q, kb, kb, table, lens[:2])
    _raises("lens must be", d, q, kb, kb, table, lens.long())
    _raises("query heads", d, _z(3, 3, 64, dtype=bf), kb, kb, table, lens)
    _raises("scale", d, q, kb, kb, table, lens, scale=0.0)
    _raises("workspace", d, q, kb, kb, table, lens, workspace=_z(16))
    _raises("out has", d, q, kb, kb, table, lens, out=q[:2])
    _raises("out overlaps q", d, q, kb, kb, table, lens, out=q)
    p = mx.mx_attn_prefill
    o = torch.tensor([0, 3], dtype=i32, device="cuda")
    _raises("v has shape", p, q, rows, rows[:2], o, o)
    _raises("k has shape", p, q, _z(3, 2, 128, dtype=bf), rows, o, o)
    _raises("q_offsets must hold", p, q, rows, rows, o[:0], o)
    _raises("k_offsets has", p, q, rows, rows, o, o[:1])
    _raises("q_offsets must be", p, q, rows, rows, o.long(), o)
    _raises("D = 32", p, _z(3, 4, 32, dtype=bf), _z(3, 2, 32, dtype=bf), _z(3, 2, 32, dtype=bf), o, o)
    _raises("out overlaps", p, rows, rows.clone(), rows, o, o, out=rows)
    torch.cuda.synchronize()


def test_shared_pages_and_one_table_for_all():
    """Sequences that share their first pages, and a head that is broadcast: the same page many times."""
    rng = np.random.default_rng(9)
    lens, D = [100, 90, 64, 17], 128
    c, table = make_cache(rng, lens, 1, D, 16, True)
    table[1:, :4] = table[0, :4]
    table[3, :2] = table[0, 1]
    q = normal(rng, 4, 6, D)
    say("shared pages")
    out = mx.mx_attn_decode(on_gpu(q), on_gpu(c["k"]), on_gpu(c["v"]), _i32(table), _i32(lens), k_scale=on_gpu(c["ks"]),
                            v_scale=on_gpu(c["vs"]))
    torch.cuda.synchronize()
    check(host_u16(out), *decode_oracle(q, c, table, lens, D ** -0.5), D, 100)


@pytest.mark.parametrize("exponent", [0, 40, -60, -130])
def test_decode_queries_of_all_magnitudes(exponent):
    """Latent rows of 512 in MXFP8, whose queries the kernel splits into two MXFP8 numbers: elements of one block spread over
    2^30, blocks of zeros, the range's ends.  An element below 2^-14 of its block's largest is off by up to 2^-21 of that; a
    weight moves by the scores' error, and the weights' sum too, so that the bound gains 2 err size."""
    rng = np.random.default_rng(10)
    H, D, lens = 48, 512, [70, 1, 300]
    c, table = make_cache(rng, lens, 1, D, 16, True, True)
    x = rng.standard_normal((3, H, D)) * 2.0 ** rng.integers(-30, 1, (3, H, D))
    x[:, ::3] = rng.standard_normal((3, H // 3, D)) * 2.0 ** rng.integers(-8, 1, (3, H // 3, D))
    x[:, 1, 64:96] = 0
    x[:, 2] = 0
    q = workloads.to_bf16_bits((x * 2.0 ** exponent).astype(np.float32))
    scale = D ** -0.5 * 2.0 ** min(-exponent, 100)
    say("decode all magnitudes", exponent)
    out = mx.mx_attn_decode(on_gpu(q), on_gpu(c["k"]), None, _i32(table), _i32(lens), k_scale=on_gpu(c["ks"]), scale=scale)
    torch.cuda.synchronize()
    ref, size, spread = decode_oracle(q, c, table, lens, scale)
    qf = F.bf16_to_f64(q).reshape(3, H, D // 32, 32)
    for b, n in enumerate(lens):
        k = np.abs(A.sequence(c["k"], c["ks"], table[b], n)).reshape(n, D // 32, 32).sum(-1).max(0)      # a block's largest sum
        err = scale * 2.0 ** -21 * (np.abs(qf[b]).max(-1) * k).sum(-1)
        spread[b] += err * 2.0 ** 24 / (D + 4)
    check(host_u16(out), ref, size, spread, D, max(lens))


@pytest.mark.parametrize("G,D,latent", [(4, 128, False), (40, 128, False), (64, 512, True), (3, 512, False)])
@pytest.mark.parametrize("what", [0x7F80, 0xFF80, 0x7FC0])
@KINDS
def test_queries_that_are_not_finite(G, D, latent, what, fp8):
    """An infinity or NaN in a head's query makes that head NaN, and no other."""
    rng = np.random.default_rng(G)
    lens = [300, 1]
    c, table = make_cache(rng, lens, 1, D, 16, fp8, latent)
    q = normal(rng, 2, G, D)
    q[0, 1, 37], q[1, G - 1, D - 1], q[1, 0, 0] = what, what, what
    say("query not finite", G, D, latent, hex(what), fp8)
    out = mx.mx_attn_decode(on_gpu(q), on_gpu(c["k"]), on_gpu(c["v"]), _i32(table), _i32(lens), k_scale=on_gpu(c["ks"]),
                            v_scale=on_gpu(c["vs"]))
    keys = normal(rng, 400, 1, D)
    dk = on_gpu(keys)
    pre = mx.mx_attn_prefill(on_gpu(q), dk, dk, _i32([0, 2]), _i32([0, 400]))
    torch.cuda.synchronize()
    bad = np.zeros((2, G), bool)
    bad[0, 1] = bad[1, G - 1] = bad[1, 0] = True
    for got in (host_u16(out), host_u16(pre)):
        f = F.bf16_to_f64(got)
        assert np.isnan(f[bad]).all() and np.isfinite(f[~bad]).all()


@pytest.mark.parametrize("G", [1, 5, 17, 33])
def test_decode_latent_bf16_of_few_heads_in_parts(G):
    """Any number of heads over a latent BF16 row of 512, streams that are cut into parts and ones that are not."""
    rng = np.random.default_rng(G)
    lens = [2000, 0, 3, 129, 700]
    c, table = make_cache(rng, lens, 1, 512, 32, False, True)
    q = normal(rng, len(lens), G, 512)
    say("decode latent bf16", G)
    out = mx.mx_attn_decode(on_gpu(q), on_gpu(c["k"]), None, _i32(table), _i32(lens))
    torch.cuda.synchronize()
    check(host_u16(out), *decode_oracle(q, c, table, lens, 512 ** -0.5), 512, 2000)


# --------------------------------------- shares of many tiles, long histories

def _shares(rng, B, Hkv, G, D, page, fp8, latent, tile, groups, tiles, heads):
    """Enough tokens for shares of `tiles` tiles in every one of `groups` groups: shares that end one stream, pass empty sequences and
    begin another, several in one stream, and one that its stream does not fill.  Scores have a deviation of 3, so that a
    sequence's output is that of few of its keys, and a tile that is left out or counted twice shows."""
    lens = spread_lens(rng, B, int(tiles * groups * tile / Hkv * 1.1))
    c, table = random_cache(rng, lens, Hkv, D, page, fp8, latent)
    H = Hkv * G
    q = normal(rng, B, H, D)
    some = A.values(c["k"][0], None if c["ks"] is None else c["ks"][0])
    scale = 3 / float(np.sqrt(D * np.mean(some ** 2)))
    ws = torch.zeros(mx.mx_attn_decode_workspace_bytes(B, H, Hkv, D, table.shape[1], page), dtype=torch.uint8, device="cuda")
    say("decode shares", B, Hkv, G, D, page, fp8, latent, sum(lens), max(lens))
    out = mx.mx_attn_decode(on_gpu(q), on_gpu(c["k"]), on_gpu(c["v"]), _i32(table), _i32(lens), k_scale=on_gpu(c["ks"]),
                            v_scale=on_gpu(c["vs"]), scale=scale, workspace=ws)
    torch.cuda.synchronize()
    assert int(ws[:4].view(torch.int32)) >= tiles                   # the plan begins with the share
    got = host_u16(out)
    assert not got[np.array(lens) == 0].any() and np.isfinite(F.bf16_to_f64(got)).all()
    check(got[:, heads], *sampled_oracle(q, c, table, lens, scale, heads), D, max(lens))


@pytest.mark.parametrize("B,Hkv,G,D,fp8,latent", [(70, 8, 4, 128, True, False), (300, 8, 2, 64, True, False), (300, 4, 3, 128, False, False),
                                                  (70, 8, 5, 64, False, False), (70, 6, 5, 256, True, False), (300, 4, 2, 256, False, False),
                                                  (70, 2, 17, 128, True, False), (70, 2, 3, 512, True, False), (70, 2, 3, 512, False, False),
                                                  (300, 1, 16, 512, True, True)])
def test_decode_shares_of_several_tiles(B, Hkv, G, D, fp8, latent):
    rng = np.random.default_rng(B + G + D)
    groups = (512 if D < 512 else 256) // -(-G // 16)
    heads = sorted({0, G - 1, Hkv * G // 2, Hkv * G - 1, *(int(h) for h in rng.integers(0, Hkv * G, 4))})
    _shares(rng, B, Hkv, G, D, 64, fp8, latent, 128, groups, 3, heads)


@pytest.mark.parametrize("B,Hkv,G,D,fp8,latent", [(70, 2, 40, 128, True, False), (300, 1, 130, 64, True, False), (70, 1, 130, 64, False, False),
                                                  (70, 1, 130, 128, False, True), (70, 1, 40, 256, True, True), (70, 1, 130, 256, False, False),
                                                  (300, 1, 33, 512, True, True), (70, 1, 128, 512, True, True), (70, 1, 128, 512, False, True),
                                                  (300, 1, 4, 512, False, True)])
def test_decode_shares_of_many_tiles_with_heads_as_rows(B, Hkv, G, D, fp8, latent):
    rng = np.random.default_rng(B + G + D)
    groups = (512 if D < 512 else 256) // -(-G // 128)
    heads = sorted({0, G - 1, min(127, G - 1), Hkv * G - 1, *(int(h) for h in rng.integers(0, Hkv * G, 3))})
    _shares(rng, B, Hkv, G, D, 32, fp8, latent, 64 if D <= 128 else 32, groups, 9, heads)


@pytest.mark.parametrize("lens,past,Hkv,G", [([200, 1], [9000, 5003], 2, 2), ([3, 7, 1], [8001, 30, 6000], 1, 5), ([1300], [77], 1, 1)])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("same", [False, True])
def test_prefill_over_long_keys(lens, past, Hkv, G, D, same):
    """Keys split over workgroups, many tiles in each split, and rows that are not split."""
    _prefill(np.random.default_rng(sum(lens) + D), lens, past, Hkv, G, D, same=same)


@pytest.mark.parametrize("H", [40, 130])
def test_decode_queries_at_the_top_of_the_range(H):
    """The same split of queries up to the largest BF16 number, whose nearest MXFP8 number is 2^128, over keys so small that
    scores are about 1: scores and outputs are as finite as the formula's, bounds as above."""
    rng = np.random.default_rng(11)
    D, lens = 512, [70, 1, 300]
    c, table = make_cache(rng, lens, 1, D, 16, True, True)
    c["ks"] -= 20                                                   # keys times 2^-20
    x = rng.integers(0x7F00, 0x7F80, (3, H, D)) | (rng.integers(0, 2, (3, H, D)) << 15)      # 2^127 and above, either sign
    x[:, 1] = np.where(rng.random((3, D)) < 0.5, 0x7F7F, 0xFF7F)
    x[:, 2, 1::2] -= 0x0300                                         # and times 2^-6 between them
    x[:, 3, :] -= 0x0100                                            # the next powers of two down
    x[:, 4, :] -= 0x0080
    q = x.astype(np.uint16)
    scale = D ** -0.5 * 2.0 ** -107
    say("decode top of the range", H)
    out = mx.mx_attn_decode(on_gpu(q), on_gpu(c["k"]), None, _i32(table), _i32(lens), k_scale=on_gpu(c["ks"]), scale=scale)
    torch.cuda.synchronize()
    ref, size, spread = decode_oracle(q, c, table, lens, scale)
    assert np.isfinite(ref).all() and spread.max() < 64
    qf = F.bf16_to_f64(q).reshape(3, H, D // 32, 32)
    for b, n in enumerate(lens):
        k = np.abs(A.sequence(c["k"], c["ks"], table[b], n)).reshape(n, D // 32, 32).sum(-1).max(0)      # a block's largest sum
        err = scale * 2.0 ** -21 * (np.abs(qf[b]).max(-1) * k).sum(-1)
        spread[b] += err * 2.0 ** 24 / (D + 4)
    check(host_u16(out), ref, size, spread, D, max(lens))


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_prefill_splits_of_512_keys_at_least(D):
    """Rows that see 512 keys or fewer are not split: their parts of the workspace, [row tile][split] of 128 rows, stay as they were;
    rows that see 1024 leave two parts, whatever the head's size."""
    rng = np.random.default_rng(D)
    rows = 1024
    q, k, v = (on_gpu(normal(rng, rows, 1, D)) for _ in range(3))
    offsets = _i32([0, rows])
    need = mx.mx_attn_prefill_workspace_bytes(1, rows, rows, 1, 1, D)
    part = 128 * (D + 2) * 4
    assert need >= 9 * 2 * part
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    say("prefill least split", D)
    mx.mx_attn_prefill(q, k, v, offsets, offsets, workspace=ws)
    torch.cuda.synchronize()
    parts = host_u8(ws)[:9 * 2 * part].reshape(9, 2, part)
    assert (parts[:4] == 0xFF).all() and (parts[8] == 0xFF).all()
    assert (parts[4:8, :, -128 * 4:] != 0xFF).any(-1).all()


# ------------------------------------------- nothing to do, and replays

@KINDS
def test_nothing_to_do(fp8):
    """No tokens, no sequences, no rows, no keys: outputs of that many rows, and rows without keys are 0."""
    rng = np.random.default_rng(12)
    Hkv, H, D = 2, 4, 128
    c, table = make_cache(rng, [20, 5], Hkv, D, 16, fp8)
    k, v, ks, vs = (on_gpu(c[n]) for n in ("k", "v", "ks", "vs"))
    kept = [t.clone() for t in (k, v, ks, vs) if t is not None]
    none = torch.zeros((0, Hkv, D), dtype=torch.bfloat16, device="cuda")
    q = on_gpu(normal(rng, 7, H, D)).view(torch.bfloat16)
    say("nothing to do", fp8)
    mx.mx_kv_cache_write(none, none, dev_i64([]), k, v, k_scale=ks, v_scale=vs)
    mx.mx_kv_cache_write(q[:3, :2], q[:3, 2:], dev_i64([-1, -1, 1 << 40]), k, v, k_scale=ks, v_scale=vs)
    kk, vv = mx.mx_kv_cache_read(k, v, _i32(table[:0]), _i32([0]), 0, k_scale=ks, v_scale=vs)
    k0, v0 = mx.mx_kv_cache_read(k, v, _i32(table), _i32([0, 0, 0]), 0, k_scale=ks, v_scale=vs)
    assert all(t.shape == (0, Hkv, D) for t in (kk, vv, k0, v0))
    assert mx.mx_attn_decode(q[:0], k, v, _i32(table[:0]), _i32([]), k_scale=ks, v_scale=vs).shape == (0, H, D)
    assert mx.mx_attn_prefill(q[:0], none, none, _i32([0, 0]), _i32([0, 0])).shape == (0, H, D)
    assert mx.mx_attn_prefill(q[:0], none, none, _i32([0]), _i32([0])).shape == (0, H, D)
    zero = [mx.mx_attn_prefill(q, none, none, _i32([0, 3, 7]), _i32([0, 0, 0])), mx.mx_attn_prefill(q, none, none.clone(), _i32([0, 3, 7]), _i32([0, 0, 0])),
            mx.mx_attn_decode(q[:2], k, v, _i32(table), _i32([0, -3]), k_scale=ks, v_scale=vs)]
    torch.cuda.synchronize()
    assert all(not t.view(torch.int16).any() for t in zero)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(kept, (t for t in (k, v, ks, vs) if t is not None)))


@pytest.mark.parametrize("D,G,latent", [(512, 128, True), (512, 5, True), (128, 40, False), (256, 4, False)])
@KINDS
def test_graph_of_shares(D, G, latent, fp8):
    """Captured once and replayed over other lengths, with empty sequences among them and eager calls between: every replay equals
    the eager call."""
    rng = np.random.default_rng(13)
    B, page = 5, 32
    c, table = make_cache(rng, [1500] * B, 1, D, page, fp8, latent)
    k, v, ks, vs = (on_gpu(c[n]) for n in ("k", "v", "ks", "vs"))
    t, lens, q = _i32(table), _i32([1500, 0, 3, 700, 64]), on_gpu(normal(rng, B, G, D))
    call = lambda: mx.mx_attn_decode(q, k, v, t, lens, k_scale=ks, v_scale=vs)  # noqa: E731
    say("graph of shares", D, G, latent, fp8)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = call()
    for at in ([1500, 0, 3, 700, 64], [0, 0, 0, 0, 1], [1, 1500, 1500, 0, 33], [0] * 5, [1500] * 5):
        lens.copy_(_i32(at))
        q.copy_(on_gpu(normal(rng, B, G, D)))
        g.replay()
        torch.cuda.synchronize()
        got = held.clone()
        want = call()
        torch.cuda.synchronize()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)), at
        assert not got[np.array(at) == 0].view(torch.int16).any() and torch.isfinite(got.float()).all()
