"""Argument checks of the key-value cache and the attention calls, on the CPU: the C entry points in dry-run mode, overlaps
outside it, workspace sizes, and the binding's shape and type checks (which run before any pointer is taken)."""

import os

import pytest
import torch

import mx_scaled_fp8_amd as mx

pytestmark = pytest.mark.skipif(not os.path.exists(mx.lib_path()), reason="libmxfp8.so not built")

FAKE = 1 << 20      # a 16-byte aligned stand-in for a device pointer; nothing is read in dry-run mode


@pytest.fixture
def dry():
    mx.mx_set_dry_run(True)
    yield
    mx.mx_set_dry_run(False)


def _refused(call, cases):
    for bad in cases:
        assert call(**bad) == mx.MX_ERR_INVALID_ARG, bad
        assert mx.lib().mx_last_error().decode()


def _write(**kw):
    a = dict(k=FAKE, ks=512, v=FAKE, vs=1024, T=100, Hkv=4, D=128, slots=FAKE, kind=0, kc=FAKE, kcs=FAKE, vc=FAKE, vcs=FAKE,
             pages=10, page=64)
    a.update(kw)
    return mx.lib().mx_kv_cache_write(*a.values(), None)


# what is wrong with a cache, in each call's names
BAD_CACHES = [dict(kind=2), dict(kind=-1), dict(kind=1), dict(kc=None), dict(kcs=None), dict(vcs=None), dict(vc=None), dict(pages=0),
              dict(pages=1 << 31), dict(pages=-1), dict(page=8), dict(page=48), dict(page=8192), dict(page=0), dict(page=-64),
              dict(Hkv=0), dict(kc=FAKE + 8), dict(kcs=FAKE + 8), dict(vc=FAKE + 4), dict(vcs=FAKE + 1),
              dict(pages=(1 << 31) - 1, page=4096)]


def test_write_validation(dry):
    assert _write() == mx.MX_OK
    assert _write(kind=1, kcs=None, vcs=None) == mx.MX_OK
    assert _write(v=None, vs=0, vc=None, vcs=None) == mx.MX_OK                       # a latent cache
    assert _write(T=0, k=None, v=None, slots=None, ks=0, vs=0) == mx.MX_OK
    for D in (32, 96, 1024):
        assert _write(D=D, ks=4 * D, vs=4 * D) == mx.MX_OK
    for page in (16, 4096):
        assert _write(page=page) == mx.MX_OK
    assert _write(T=1 << 24, Hkv=1, D=1024, ks=1024) == mx.MX_ERR_INVALID_ARG        # 2^34 elements
    _refused(_write, BAD_CACHES + [dict(D=16), dict(D=120), dict(D=1056), dict(Hkv=8193), dict(T=-1), dict(T=1 << 31), dict(k=None),
                                   dict(v=None), dict(slots=None), dict(ks=504), dict(ks=516), dict(vs=508), dict(vs=1 << 31),
                                   dict(k=FAKE + 2), dict(v=FAKE + 8), dict(slots=FAKE + 4), dict(vc=None, vcs=None)])


def _read(**kw):
    a = dict(kind=0, kc=FAKE, kcs=FAKE, vc=FAKE, vcs=FAKE, pages=10, page=64, Hkv=4, D=128, table=FAKE, B=3, max_pages=7,
             offsets=FAKE, rows=100, k=FAKE, v=FAKE)
    a.update(kw)
    return mx.lib().mx_kv_cache_read(*a.values(), None)


def test_read_validation(dry):
    assert _read() == mx.MX_OK
    assert _read(kind=1, kcs=None, vcs=None) == mx.MX_OK
    assert _read(vc=None, vcs=None, v=None) == mx.MX_OK
    assert _read(B=0, table=None, offsets=None, k=None, v=None) == mx.MX_OK
    assert _read(rows=0, table=None, offsets=None, k=None, v=None) == mx.MX_OK
    _refused(_read, BAD_CACHES + [dict(B=-1), dict(B=1 << 31), dict(rows=-1), dict(rows=1 << 31), dict(rows=1 << 28, Hkv=1, D=32), dict(rows=1 << 25), dict(max_pages=0),
                                  dict(max_pages=1 << 31), dict(k=None), dict(v=None), dict(table=None), dict(offsets=None),
                                  dict(k=FAKE + 8), dict(v=FAKE + 8), dict(table=FAKE + 2), dict(offsets=FAKE + 1), dict(D=48)])


def _decode(**kw):
    a = dict(q=FAKE, qs=1024, B=5, H=8, Hkv=4, D=128, kind=0, kc=FAKE, kcs=FAKE, vc=FAKE, vcs=FAKE, pages=10, page=64, table=FAKE,
             max_pages=7, lens=FAKE, scale=0.1, out=FAKE, ws=FAKE, wb=1 << 40)
    a.update(kw)
    return mx.lib().mx_attn_decode(*a.values(), None)


def test_decode_validation(dry):
    assert _decode() == mx.MX_OK
    assert _decode(kind=1, kcs=None, vcs=None) == mx.MX_OK
    assert _decode(vc=None, vcs=None) == mx.MX_OK
    assert _decode(B=0, q=None, table=None, lens=None, out=None, ws=None, wb=0) == mx.MX_OK
    for D in (64, 256, 512):
        assert _decode(D=D, qs=8 * D) == mx.MX_OK
    need = mx.mx_attn_decode_workspace_bytes(5, 8, 4, 128, 7, 64)
    assert need and _decode(wb=need) == mx.MX_OK
    nan, inf = float("nan"), float("inf")
    _refused(_decode, BAD_CACHES + [dict(D=96), dict(D=1024, qs=8192), dict(H=6), dict(H=0), dict(H=65540), dict(B=-1), dict(B=1 << 24),
                                    dict(B=1 << 21), dict(B=1 << 20), dict(scale=0.0), dict(scale=-1.0), dict(scale=nan), dict(scale=inf),
                                    dict(max_pages=0), dict(max_pages=1 << 31), dict(max_pages=1 << 25), dict(q=None), dict(table=None),
                                    dict(lens=None), dict(out=None), dict(qs=1016), dict(qs=1028), dict(qs=1 << 31), dict(q=FAKE + 2),
                                    dict(out=FAKE + 8), dict(table=FAKE + 2), dict(lens=FAKE + 2), dict(ws=None), dict(ws=FAKE + 8),
                                    dict(wb=need - 1), dict(B=1 << 16, max_pages=1 << 20)])


def _prefill(**kw):
    a = dict(q=FAKE, qs=1024, k=FAKE, ks=512, v=FAKE, vs=512, qo=FAKE, ko=FAKE, B=3, Tq=1000, Tk=3000, H=8, Hkv=4, D=128, scale=0.1,
             out=FAKE, ws=FAKE, wb=1 << 40)
    a.update(kw)
    return mx.lib().mx_attn_prefill(*a.values(), None)


def test_prefill_validation(dry):
    assert _prefill() == mx.MX_OK
    assert _prefill(B=0, q=None, k=None, v=None, qo=None, ko=None, out=None, ws=None, wb=0) == mx.MX_OK
    assert _prefill(Tq=0, q=None, qo=None, ko=None, out=None, ws=None, wb=0) == mx.MX_OK
    assert _prefill(Tk=0, k=None, v=None, ks=0, vs=0) == mx.MX_OK
    for D in (64, 256, 512):
        assert _prefill(D=D, qs=8 * D, ks=4 * D, vs=4 * D) == mx.MX_OK
    need = mx.mx_attn_prefill_workspace_bytes(1, 64, 30000, 8, 4, 128)
    split = dict(B=1, Tq=64, Tk=30000)
    assert need and _prefill(**split, wb=need) == mx.MX_OK
    nan, inf = float("nan"), float("inf")
    _refused(_prefill, [dict(D=32), dict(D=96), dict(H=6), dict(H=0), dict(Hkv=0), dict(Hkv=-4), dict(H=65540), dict(B=-1), dict(B=1 << 24),
                        dict(Tq=-1), dict(Tq=1 << 31), dict(Tk=-1), dict(Tk=1 << 31), dict(Tk=(1 << 31) - 64), dict(Tq=1 << 30), dict(scale=0.0),
                        dict(scale=nan), dict(scale=inf), dict(q=None), dict(k=None), dict(v=None), dict(qo=None), dict(ko=None),
                        dict(out=None), dict(qs=1016), dict(qs=1028), dict(qs=1 << 31), dict(ks=504), dict(ks=516), dict(ks=1 << 22),
                        dict(vs=504), dict(vs=516), dict(vs=1 << 22), dict(q=FAKE + 8), dict(k=FAKE + 8), dict(v=FAKE + 8),
                        dict(out=FAKE + 8), dict(qo=FAKE + 2), dict(ko=FAKE + 2), dict(split, wb=need - 1), dict(split, ws=None),
                        dict(split, ws=FAKE + 8)])


def test_workspace_sizes():
    d, p = mx.mx_attn_decode_workspace_bytes, mx.mx_attn_prefill_workspace_bytes
    for bad in ((0, 8, 4, 128, 7, 64), (5, 3, 4, 128, 7, 64), (5, 8, 0, 128, 7, 64), (5, 8, 4, 0, 7, 64), (5, 8, 4, 128, 0, 64),
                (5, 8, 4, 128, 7, 0), (1 << 62, 8, 4, 128, 7, 64), (5, 8, 4, 128, 1 << 62, 64), (5, 1 << 30, 4, 128, 7, 64),
                (5, 8, 4, 128, 7, 1 << 30)):
        assert d(*bad) == 0, bad
    for bad in ((0, 10, 10, 8, 4, 128), (1, 0, 10, 8, 4, 128), (1, 10, -1, 8, 4, 128), (1, 10, 10, 3, 4, 128), (1, 10, 10, 8, 0, 128),
                (1 << 62, 10, 10, 8, 4, 128), (1, 1 << 62, 10, 8, 4, 128), (1, 10, 1 << 62, 8, 4, 128), (1, 10, 10, 1 << 30, 4, 128)):
        assert p(*bad) == 0, bad
    # bounded whatever the length: what is in the workspace are parts of as many workgroups as fill the card
    assert d(1, 128, 1, 512, 1 << 18, 64) < 1 << 30 and d(512, 64, 8, 128, 1 << 10, 64) < 1 << 30
    assert p(1, 64, 1 << 24, 128, 1, 512) < 1 << 30
    assert p(8, 8192, 8192, 64, 8, 128) == 0                                         # enough rows: nothing is split


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="stand-in pointers must reach no GPU")


def _overlaps(call, sizes, written, **sized):
    """Back to back, a call gets as far as asking for the device; any two parts of which one is written overlap."""
    at, places = FAKE, {}
    for n, size in sizes.items():
        places[n] = at
        at += -(-size // 16) * 16
    assert call(**dict(places, **sized)) == mx.MX_ERR_UNSUPPORTED
    for a in written:
        for b in sizes:
            if a == b:
                continue
            for place in (places[b], places[b] + (sizes[b] - 1) // 16 * 16):
                assert call(**dict(places, **sized, **{a: place})) == mx.MX_ERR_INVALID_ARG, (a, b)
                assert "overlaps" in mx.lib().mx_last_error().decode()


@no_gpu
def test_overlaps_are_refused():
    cache = dict(kc=10 * 64 * 512, vc=10 * 64 * 512, kcs=10 * 64 * 16, vcs=10 * 64 * 16)
    _overlaps(_write, dict(cache, k=(99 * 512 + 512) * 2, v=(99 * 1024 + 512) * 2, slots=800), cache)
    out = dict(k=100 * 512 * 2, v=100 * 512 * 2)
    _overlaps(_read, dict(out, **cache, table=3 * 7 * 4, offsets=16), out)
    need = mx.mx_attn_decode_workspace_bytes(5, 8, 4, 128, 7, 64)
    out = dict(out=5 * 1024 * 2, ws=need)
    _overlaps(_decode, dict(out, q=5 * 1024 * 2, **cache, table=5 * 7 * 4, lens=20), out, wb=need)
    need = mx.mx_attn_prefill_workspace_bytes(1, 64, 30000, 8, 4, 128)
    out = dict(out=64 * 1024 * 2, ws=need)
    _overlaps(_prefill, dict(out, q=64 * 1024 * 2, k=30000 * 1024, v=30000 * 1024, qo=8, ko=8), out, wb=need, B=1, Tq=64, Tk=30000)


# ------------------------------------------------------------- the binding

i16, i32, i64, u8 = torch.int16, torch.int32, torch.int64, torch.uint8


def z(*shape, dtype=u8):
    return torch.zeros(shape, dtype=dtype)


def _raises(match, f, *a, **kw):
    with pytest.raises((ValueError, TypeError), match=match):
        f(*a, **kw)


def test_binding_wants_gpu_tensors():
    kc, sc = z(4, 2, 16, 64), z(4, 2, 16, 2)
    rows = z(3, 2, 64, dtype=i16)
    _raises("k must be a GPU tensor", mx.mx_kv_cache_write, rows, rows, z(3, dtype=i64), kc, kc, sc, sc)
    _raises("k_cache must be a GPU tensor", mx.mx_kv_cache_read, kc, kc, z(1, 2, dtype=i32), z(2, dtype=i32), 3, sc, sc)
    _raises("q must be a GPU tensor", mx.mx_attn_decode, z(1, 4, 64, dtype=i16), kc, kc, z(1, 2, dtype=i32), z(1, dtype=i32), sc, sc)
    _raises("q must be a GPU tensor", mx.mx_attn_prefill, rows, rows, rows, z(2, dtype=i32), z(2, dtype=i32))
    _raises("k must be a torch tensor", mx.mx_kv_cache_write, [1], rows, z(3, dtype=i64), kc, kc, sc, sc)


def test_sizes_that_a_call_refuses_have_no_workspace(dry):
    """The queries are public and come before the call that refuses: one of them divided by a product that had wrapped to 0."""
    d, p = mx.mx_attn_decode_workspace_bytes, mx.mx_attn_prefill_workspace_bytes
    for B, Tq, Tk, H, Hkv, D in ((1 << 23, (1 << 24) - (1 << 14), 1 << 20, 65536, 1, 128), ((1 << 24) - 1, (1 << 31) - 1, 100, 65536, 1, 64),
                                 (1, 100, 100, 6, 4, 128), (1, 100, 100, 8, 4, 96), (1, 1 << 30, 100, 8, 4, 128)):
        assert p(B, Tq, Tk, H, Hkv, D) == 0
        assert _prefill(B=B, Tq=Tq, Tk=Tk, H=H, Hkv=Hkv, D=D, qs=H * D, ks=Hkv * D, vs=Hkv * D) == mx.MX_ERR_INVALID_ARG
    for B, H, Hkv, D, n, page in (((1 << 24) - 1, 65536, 65536, 512, 1 << 18, 4096), (5, 6, 4, 128, 7, 64), (5, 8, 4, 96, 7, 64),
                                  (5, 8, 4, 128, 7, 48), (1 << 20, 8, 4, 128, 7, 64), (1, 4096, 4096, 512, 7, 64)):
        assert d(B, H, Hkv, D, n, page) == 0
        assert _decode(B=B, H=H, Hkv=Hkv, D=D, max_pages=n, page=page, qs=H * D) == mx.MX_ERR_INVALID_ARG


def test_read_of_as_many_rows_as_a_launch_has_threads_for(dry):
    """16 rows to a workgroup of 256 threads: 2^28 - 15 rows would be 2^32 threads."""
    assert _read(rows=(1 << 28) - 16, Hkv=1, D=32) == mx.MX_OK
    _refused(_read, [dict(rows=(1 << 28) - 15, Hkv=1, D=32), dict(rows=(1 << 28) - 1, Hkv=1, D=32)])


def test_scales_that_leave_fp32_in_powers_of_two(dry):
    """The kernels take scale * log2(e): infinite, it would make NaN of scores of 0."""
    for call in (_decode, _prefill):
        assert call(scale=2.0 ** 127) == mx.MX_OK and call(scale=2.0 ** -149) == mx.MX_OK
        _refused(call, [dict(scale=2.4e38), dict(scale=3.4e38), dict(scale=1e39), dict(scale=-2.0 ** -149)])


@pytest.mark.parametrize("D,groups", [(64, 512), (128, 512), (256, 256), (512, 256)])
def test_parts_of_as_many_groups_as_run_at_once(D, groups):
    """Two workgroups on each of 256 compute units, one of heads of 256 and more; a group leaves two parts of 16 heads (O, m, l) behind
    the plan."""
    assert mx.mx_attn_decode_workspace_bytes(63, 16, 4, D, 128, 64) == 64 * 4 + groups * 2 * 16 * (D + 2) * 4
