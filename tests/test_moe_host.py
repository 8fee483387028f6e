"""Argument checks of the mixture-of-experts calls and the block-128 linear, on the CPU: the C entry points in dry-run
mode, and the binding's shape and type checks (which run before any pointer is taken)."""

import os

import pytest
import torch

import mx_scaled_fp8_amd as mx

pytestmark = pytest.mark.skipif(not os.path.exists(mx.lib_path()), reason="libmxfp8.so not built")

FAKE = 1 << 20      # a 16-byte aligned stand-in for a device pointer; nothing is read in dry-run mode
BIG = 1 << 44       # another, far from it


@pytest.fixture
def dry():
    mx.mx_set_dry_run(True)
    yield
    mx.mx_set_dry_run(False)


def _route(**kw):
    a = dict(logits=FAKE, f32=1, bias=FAKE, T=100, E=64, k=8, score=0, renorm=1, scale=1.0, ids=FAKE, weights=FAKE,
             offsets=FAKE, row_slot=FAKE, slot_row=FAKE, ws=FAKE, wb=1 << 30)
    a.update(kw)
    return mx.lib().mx_moe_route(*a.values(), None)


def test_route_validation(dry):
    assert _route() == mx.MX_OK
    assert _route(bias=None) == mx.MX_OK
    assert _route(f32=0, logits=FAKE + 2) == mx.MX_OK                # BF16 logits
    assert _route(T=0, logits=None, ids=None, weights=None, row_slot=None, slot_row=None, ws=None, wb=0) == mx.MX_OK
    assert _route(T=64, ws=None, wb=0) == mx.MX_OK                   # one block of tokens needs no workspace
    assert _route(E=1, k=1) == mx.MX_OK
    assert _route(E=1024, k=32) == mx.MX_OK
    need = mx.mx_moe_route_workspace_bytes(100, 64)
    assert need == 4 * 64 * (8 + 1) and _route(wb=need) == mx.MX_OK
    for bad in (dict(f32=2), dict(E=0), dict(E=1025), dict(k=0), dict(k=65), dict(E=4, k=5), dict(k=33), dict(T=-1),
                dict(T=1 << 30), dict(T=1 << 29, E=2, k=1), dict(score=2), dict(renorm=2), dict(logits=None), dict(ids=None), dict(weights=None),
                dict(offsets=None), dict(row_slot=None), dict(slot_row=None), dict(logits=FAKE + 2),
                dict(offsets=FAKE + 2), dict(ws=None), dict(ws=FAKE + 4), dict(wb=need - 1), dict(bias=FAKE + 1)):
        assert _route(**bad) == mx.MX_ERR_INVALID_ARG, bad
        assert mx.lib().mx_last_error().decode()


no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="stand-in pointers must reach no GPU")


@no_gpu
def test_route_refuses_tensors_that_overlap():
    """Outside a dry run, before any device is asked for: a call of tensors that lie apart gets as far as that."""
    T, E, k = 100, 64, 8
    names = ("logits", "bias", "ids", "weights", "offsets", "row_slot", "slot_row", "ws")
    size = dict(logits=T * E * 4, bias=E * 4, offsets=(E + 1) * 4, ws=mx.mx_moe_route_workspace_bytes(T, E))
    size.update((n, T * k * 4) for n in ("ids", "weights", "row_slot", "slot_row"))
    at, places = FAKE, {}
    for n in names:                                                  # back to back
        places[n] = at
        at += -(-size[n] // 8) * 8
    assert _route(T=T, E=E, k=k, **places) == mx.MX_ERR_UNSUPPORTED
    for a in names:
        for b in names:
            if a == b or {a, b} == {"logits", "bias"}:
                continue
            for place in (places[b], places[b] + (size[b] - 8) // 8 * 8):
                assert _route(T=T, E=E, k=k, **dict(places, **{a: place})) == mx.MX_ERR_INVALID_ARG, (a, b)
                assert "overlaps" in mx.lib().mx_last_error().decode()
    # a bias inside the logits is read alone
    assert _route(T=T, E=E, k=k, **dict(places, bias=places["logits"])) == mx.MX_ERR_UNSUPPORTED


def _grouped(**kw):
    a = dict(x=FAKE, rows=100, K=576, w=BIG, ws=FAKE, kind=0, E=8, N=512, offsets=FAKE, row_slot=FAKE, k=2, S=200,
             act=0, out=2 * BIG, work=FAKE, wb=1 << 40)
    a.update(kw)
    return mx.lib().mx_grouped_linear(*a.values(), None)


def test_grouped_validation(dry):
    assert _grouped() == mx.MX_OK
    assert _grouped(kind=1) == mx.MX_OK
    assert _grouped(kind=1, K=16) == mx.MX_OK
    assert _grouped(row_slot=None, S=100) == mx.MX_OK
    assert _grouped(S=0) == mx.MX_OK
    assert _grouped(rows=0, S=0, x=None, w=None, out=None, work=None, wb=0) == mx.MX_OK
    need = mx.mx_grouped_linear_workspace_bytes(100, 200, 8, 512, 576)
    assert need >= 100 * 640 and _grouped(wb=need) == mx.MX_OK
    for bad in (dict(kind=2), dict(act=2), dict(k=0), dict(K=0), dict(K=48), dict(kind=1, K=24), dict(K=1 << 22),
                dict(N=0), dict(N=24), dict(E=0), dict(E=1 << 20), dict(S=-1), dict(rows=-1), dict(S=1 << 31),
                dict(row_slot=None), dict(rows=0), dict(rows=1 << 30), dict(x=None), dict(w=None), dict(ws=None),
                dict(offsets=None), dict(out=None), dict(x=FAKE + 8), dict(w=BIG + 4), dict(out=2 * BIG + 8),
                dict(kind=1, ws=FAKE + 2), dict(offsets=FAKE + 2), dict(row_slot=FAKE + 1), dict(work=None),
                dict(work=FAKE + 8), dict(wb=need - 1), dict(out=BIG + 512), dict(out=FAKE),
                dict(S=(1 << 31) - 1, N=1 << 20), dict(S=1 << 29, N=256), dict(S=1 << 28, N=512),
                dict(ws=2 * BIG + 64), dict(offsets=2 * BIG + 64), dict(row_slot=2 * BIG + 64), dict(work=2 * BIG + 64)):
        assert _grouped(**bad) == mx.MX_ERR_INVALID_ARG, bad
        assert mx.lib().mx_last_error().decode()


def test_block128_validation(dry):
    def f(**kw):
        a = dict(x=FAKE, M=65, K=144, w=BIG, ws=FAKE, N=48, out=2 * BIG, work=FAKE, wb=1 << 30)
        a.update(kw)
        return mx.lib().mx_linear_block128(*a.values(), None)
    assert f() == mx.MX_OK
    assert f(M=0, x=None, out=None, work=None, wb=0) == mx.MX_OK
    need = mx.mx_linear_block128_workspace_bytes(65, 48, 144)
    assert f(wb=need) == mx.MX_OK
    for bad in (dict(M=-1), dict(K=8), dict(K=100), dict(N=8), dict(N=50), dict(x=None), dict(w=None), dict(ws=None),
                dict(out=None), dict(x=FAKE + 2), dict(w=BIG + 8), dict(ws=FAKE + 1), dict(out=2 * BIG + 8),
                dict(work=None), dict(wb=need - 1), dict(out=BIG), dict(M=1 << 26, K=4096)):
        assert f(**bad) == mx.MX_ERR_INVALID_ARG, bad


@no_gpu
@pytest.mark.parametrize("kind", [0, 1])
def test_products_refuse_a_workspace_over_an_input(kind):
    """Outside a dry run, before any device is asked for: a call of tensors that lie apart gets as far as that."""
    rows, S, K, E, N = 100, 200, 576, 8, 512
    size = dict(x=rows * K * 2, w=E * N * K, ws=E * N * (K // 32) if kind == 0 else E * 4 * 5 * 4, offsets=(E + 1) * 4,
                row_slot=S * 4, work=mx.mx_grouped_linear_workspace_bytes(rows, S, E, N, K))
    at, places = FAKE, {}
    for n, b in size.items():                                        # back to back
        places[n] = at
        at += -(-b // 16) * 16
    assert _grouped(kind=kind, **places) == mx.MX_ERR_UNSUPPORTED
    dense = lambda **p: mx.lib().mx_linear_block128(p["x"], rows, K, p["w"], p["ws"], N, 2 * BIG, p["work"], 1 << 30, None)
    assert dense(**places) == mx.MX_ERR_UNSUPPORTED
    for n in ("x", "w", "ws", "offsets", "row_slot"):
        for work in (places[n], places[n] + (size[n] - 1) // 16 * 16):
            p = dict(places, work=work)
            if n == "x":
                p["w"] = BIG                                         # so that only x is met
            assert _grouped(kind=kind, **p) == mx.MX_ERR_INVALID_ARG, n
            assert "workspace overlaps" in mx.lib().mx_last_error().decode()
            if kind == 1 and n in ("x", "w", "ws") and work == places[n]:   # the dense weight is the first expert's
                assert dense(**p) == mx.MX_ERR_INVALID_ARG, n


def test_combine_validation(dry):
    def f(**kw):
        a = dict(y=FAKE, rows=80, N=512, slot_row=FAKE, weights=FAKE, T=10, k=8, shared=BIG, out=2 * BIG)
        a.update(kw)
        return mx.lib().mx_moe_combine(*a.values(), None)
    assert f() == mx.MX_OK
    assert f(shared=None) == mx.MX_OK
    assert f(out=BIG) == mx.MX_OK                                    # in place over the shared rows
    assert f(T=0, y=None, out=None) == mx.MX_OK
    assert f(rows=0, y=None) == mx.MX_OK                             # every slot dropped
    assert f(out=FAKE + 80 * 512 * 2) == mx.MX_OK                    # behind y
    for bad in (dict(T=-1), dict(rows=-1), dict(rows=1 << 31), dict(N=0), dict(N=12), dict(k=0), dict(k=1025),
                dict(y=None), dict(slot_row=None), dict(weights=None), dict(out=None), dict(y=FAKE + 8),
                dict(out=2 * BIG + 2), dict(shared=BIG + 8), dict(slot_row=FAKE + 2), dict(out=FAKE + 1024),
                dict(out=BIG + 1024), dict(T=1 << 30, N=1 << 10), dict(T=1 << 30, N=32)):
        assert f(**bad) == mx.MX_ERR_INVALID_ARG, bad


def test_combine_refuses_out_over_the_slots(dry):
    T, k, N = 10, 8, 512
    for name in ("slot_row", "weights"):
        for at, ok in ((BIG + T * k * 4, True), (BIG + T * k * 4 - 16, False), (BIG, False), (BIG - T * N * 2 + 16, False),
                       (BIG - T * N * 2, True)):
            a = dict(y=FAKE, rows=80, N=N, slot_row=2 * BIG, weights=2 * BIG, T=T, k=k, shared=None, out=at)
            a[name] = BIG
            st = mx.lib().mx_moe_combine(*a.values(), None)
            assert st == (mx.MX_OK if ok else mx.MX_ERR_INVALID_ARG), (name, at - BIG)


def z(*shape, dtype=torch.uint8):
    return torch.zeros(shape, dtype=dtype)


def _raises(match, fn, *a, **k):
    with pytest.raises(ValueError, match=match):
        fn(*a, **k)


i16, i32, f32 = torch.int16, torch.int32, torch.float32


def test_route_binding_checks():
    l, b = z(8, 16, dtype=f32), z(16, dtype=f32)
    _raises("logits must be", mx.mx_moe_route, z(8, dtype=f32), 2)
    _raises("logits must be", mx.mx_moe_route, z(8, 16, dtype=torch.float64), 2)
    _raises("bias has", mx.mx_moe_route, l, 2, bias=z(15, dtype=f32))
    _raises("bias must be", mx.mx_moe_route, l, 2, bias=z(16, dtype=i16))
    _raises("k = 0", mx.mx_moe_route, l, 0)
    _raises("ids has", mx.mx_moe_route, l, 2, ids=z(8, dtype=i32))
    _raises("ids must be", mx.mx_moe_route, l, 2, ids=z(8, 2, dtype=torch.int64))
    _raises("weights has", mx.mx_moe_route, l, 2, weights=z(8, 3, dtype=f32))
    _raises("offsets has", mx.mx_moe_route, l, 2, offsets=z(16, dtype=i32))
    _raises("row_slot has", mx.mx_moe_route, l, 2, row_slot=z(15, dtype=i32))
    _raises("slot_row has", mx.mx_moe_route, l, 2, slot_row=z(17, dtype=i32))
    _raises("GPU tensor", mx.mx_moe_route, l, 2, bias=b)


def test_grouped_binding_checks():
    E, N, K, T, k = 4, 32, 64, 6, 2
    x, w, ws = z(T, K, dtype=i16), z(E, N, K), z(E, N, K // 32)
    off, rs = z(E + 1, dtype=i32), z(T * k, dtype=i32)
    g = mx.mx_grouped_linear
    _raises("x must be", g, z(T * K, dtype=i16), w, ws, off)
    _raises("x must be", g, z(T, K, dtype=f32), w, ws, off)
    _raises("x has shape", g, z(T, K + 32, dtype=i16), w, ws, off)
    _raises("x has shape", g, x, w, ws, off, act=mx.MX_ACT_SWIGLU)
    _raises("w_scale has shape", g, x, w, z(E, N, 1), off)
    _raises("w_scale has shape", g, x, w, z(E, 1, 2, dtype=f32), off)
    _raises("w_scale must be", g, x, w, z(E, N, 2, dtype=i16), off)
    _raises("multiple of 32", g, z(T, 48, dtype=i16), z(E, N, 48), z(E, N, 1), off)
    _raises("offsets has", g, x, w, ws, z(E, dtype=i32))
    _raises("offsets must be", g, x, w, ws, z(E + 1, dtype=torch.int64))
    _raises("row_slot must be", g, x, w, ws, off, row_slot=z(12, dtype=torch.int64), k=k)
    _raises("out has", g, x, w, ws, off, row_slot=rs, k=k, out=z(T, N, dtype=i16))
    _raises("GPU tensor", g, x, w, ws, off, row_slot=rs, k=k)


def test_combine_and_block128_binding_checks():
    T, k, N = 6, 2, 32
    y, sr, wt = z(T * k, N, dtype=i16), z(T, k, dtype=i32), z(T, k, dtype=f32)
    c = mx.mx_moe_combine
    _raises("y must be", c, z(12, dtype=i16), sr, wt)
    _raises("slot_row must be", c, y, z(T, k, dtype=torch.int64), wt)
    _raises("weights has", c, y, sr, z(T, 3, dtype=f32))
    _raises("weights must be", c, y, sr, z(T, k, dtype=i16))
    _raises("shared has", c, y, sr, wt, shared=z(T, N + 8, dtype=i16))
    _raises("out has", c, y, sr, wt, out=z(T, N + 8, dtype=i16))
    _raises("GPU tensor", c, y, sr, wt)
    x, w, ws = z(5, 144, dtype=i16), z(48, 144), z(1, 2, dtype=f32)
    b = mx.mx_linear_block128
    _raises("w has shape", b, x, z(48, 128), ws)
    _raises("w_scale has shape", b, x, w, z(1, 1, dtype=f32))
    _raises("w_scale must be", b, x, w, z(1, 2))
    _raises("out has", b, x, w, ws, out=z(5, 32, dtype=i16))
    _raises("GPU tensor", b, x, w, ws)


def test_types_of_the_same_width_are_refused():
    """An output of another 16-bit type, or a weight in another FP8 format, would be read as what it is not."""
    half = z(6, 32, dtype=torch.float16)
    x, w, off = z(6, 64, dtype=i16), z(4, 32, 64), z(5, dtype=i32)
    y, sr, wt = z(12, 32, dtype=i16), z(6, 2, dtype=i32), z(6, 2, dtype=f32)
    g, b, c = mx.mx_grouped_linear, mx.mx_linear_block128, mx.mx_moe_combine
    ws, wsf = z(4, 32, 2), z(1, 1, dtype=f32)
    _raises("out must be", g, x, w, ws, off, out=half)
    _raises("out must be", b, x, w[0], wsf, out=half)
    _raises("out must be", c, y, sr, wt, out=half)
    for t in (torch.float8_e4m3fnuz, torch.float8_e5m2, torch.bool):
        _raises("w must be", g, x, w.to(t), ws, off)
        _raises("w must be", b, x, w[0].to(t), wsf)
    for t in (torch.uint8, torch.int8, torch.float8_e4m3fn):          # OCP codes: as far as the device check
        _raises("GPU tensor", g, x, w.view(t), ws, off)
        _raises("GPU tensor", b, x, w[0].view(t), wsf)
