"""Router, grouped FP8 products, join and the block-128 linear on the GPU against the fp64 oracle.

Bounds:
* ids, offsets, row_slot, slot_row: equal.
* Router weights: a relative 2^-17.  The scores are FP32: forming l - max rounds to 2^-24 |l - max|, at most 2^-19 for
  the |l - max| <= 32 of these inputs (where larger, the weight is below e^-32 and the absolute term decides); the
  exponential, the sum over up to 1024 experts (16 in a lane, 6 steps across), two divisions and the scale add at most
  40 roundings of 2^-24, below 2^-18.
* Products: the library's bound for GEMM outputs (helpers.assert_gemm_close).  With SwiGLU the input's BF16 rounding
  may fall either way where silu(gate) * up lies within the FP32 evaluation's error of a rounding border; the product
  of the two quantised candidates' difference with |W| is added to the bound (zero nearly everywhere).
* Join: FP32 sums of k + 1 terms, each addition within 2^-24 of a partial sum that no term's magnitude sum exceeds, and
  one rounding to BF16 (2^-8, relative): 2^-8 |ref| + (k + 2) 2^-23 sum |terms|.
"""

import numpy as np
import pytest
import torch

import mx_scaled_fp8_amd as mx
import workloads
from helpers import dev_u8, dev_u16, host_u16, requires_gpu, say
from oracle import formats as F
from oracle import moe as M

pytestmark = [pytest.mark.gpu, requires_gpu, pytest.mark.timeout(300)]


def _f32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


# ------------------------------------------------------------------ router

def _check_route(l64, dev_logits, k, bias=None, score=0, renorm=True, scale=1.0):
    got = mx.mx_moe_route(dev_logits, k, bias=None if bias is None else _f32(bias), score=score, renormalize=renorm,
                          scale=scale)
    torch.cuda.synchronize()
    ids, w, off, rs, sr = [t.cpu().numpy() for t in got]
    rid, rw, roff, rrs, rsr = M.route(l64, k, bias, score, renorm, scale)
    assert np.array_equal(ids, rid)
    assert np.array_equal(off, roff) and np.array_equal(rs, rrs) and np.array_equal(sr, rsr)
    assert np.all(np.abs(w - rw) <= 2.0 ** -17 * np.abs(rw) + abs(scale) * 2.0 ** -46), np.abs(w - rw).max()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 8), (3, 5, 2), (64, 64, 6), (65, 64, 6), (1000, 65, 4), (130, 255, 8),
                                   (777, 256, 8), (40, 300, 32), (257, 512, 3), (100, 1000, 12), (2000, 1024, 1),
                                   (16, 300, 9), (17, 257, 3), (33, 129, 5), (32, 200, 16), (2049, 130, 2), (2049, 300, 4),
                                   (4097, 260, 2), (70, 100, 20), (9, 1024, 32)])
@pytest.mark.parametrize("score", [mx.MX_ROUTE_SOFTMAX, mx.MX_ROUTE_SIGMOID])
@pytest.mark.parametrize("bias", [False, True])
def test_route(T, E, k, score, bias):
    rng = np.random.default_rng(T + E + k)
    l = (2 * rng.standard_normal((T, E))).astype(np.float32)
    b = (0.2 * rng.standard_normal(E)).astype(np.float32) if bias else None
    say("route", T, E, k, score, bias)
    _check_route(l.astype(np.float64), _f32(l), k, b, score, True, 2.5)
    # BF16 logits: many equal ones
    lb = workloads.to_bf16_bits(l)
    _check_route(F.bf16_to_f64(lb), dev_u16(lb), k, b, score, False)


@pytest.mark.parametrize("T,E,k", [(70, 17, 3), (300, 32, 8), (5, 31, 16), (70, 32, 20), (9, 64, 32), (300, 128, 16),
                                   (40, 100, 17)])
@pytest.mark.parametrize("score", [mx.MX_ROUTE_SOFTMAX, mx.MX_ROUTE_SIGMOID])
@pytest.mark.parametrize("bias", [False, True])
def test_route_few_experts(T, E, k, score, bias):
    """17 to 32 experts by 16 lanes a token, and k above 16 among up to 128."""
    test_route(T, E, k, score, bias)


@pytest.mark.parametrize("T", [16384, 16385, 32769, 40000])
def test_route_many_tokens(T):
    """Both block lengths, and more blocks than workgroups of the grouping."""
    rng = np.random.default_rng(T)
    l = rng.standard_normal((T, 16)).astype(np.float32)
    say("route many", T)
    _check_route(l.astype(np.float64), _f32(l), 16 if T == 40000 else 2)


@pytest.mark.parametrize("score", [mx.MX_ROUTE_SOFTMAX, mx.MX_ROUTE_SIGMOID])
@pytest.mark.parametrize("bias", [False, True])
def test_route_masks_nan_and_equal_logits(score, bias):
    inf, E = np.inf, 70
    rng = np.random.default_rng(1)
    l = rng.standard_normal((12, E)).astype(np.float32)
    l[0] = -inf                                # nothing left
    l[1] = np.nan
    l[2] = 0.0                                 # all equal
    l[3, ::2], l[3, 1::2] = 0.0, -0.0          # equal too
    l[4, 3:] = -inf                            # fewer experts than k
    l[5, [2, 9]] = inf
    l[6, 10] = np.nan
    l[7] = np.finfo(np.float32).min            # a mask of the type's lowest value
    l[8, :] = np.finfo(np.float32).min
    l[8, 5] = 1.0
    l[9, ::3] = -inf
    l[10], l[11] = -5.0, -5.0                  # scores that FP32 cannot tell apart, few and many of them
    l[10, :20] = 15.0 + 0.01 * rng.permutation(20)
    l[11, :60] = 15.0 + 0.01 * rng.permutation(60)
    b = np.zeros(E, dtype=np.float32) if bias else None
    if bias:
        b[4], b[11], b[12] = np.nan, inf, -inf
    say("route masks", score, bias)
    for renorm in (True, False):
        _check_route(l.astype(np.float64), _f32(l), 6, b, score, renorm)


def test_route_no_tokens_writes_offsets():
    off = torch.full((9,), 7, dtype=torch.int32, device="cuda")
    ids, w, off2, rs, sr = mx.mx_moe_route(torch.empty((0, 8), device="cuda"), 2, offsets=off)
    torch.cuda.synchronize()
    assert off2 is off and off.tolist() == [0] * 9 and ids.shape == (0, 2) and rs.numel() == 0


def test_route_repeats_bit_for_bit():
    g = torch.Generator(device="cuda").manual_seed(5)
    l = torch.randn((3001, 96), generator=g, device="cuda")
    a = mx.mx_moe_route(l, 5)
    for _ in range(5):
        b = mx.mx_moe_route(l, 5)
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("E", [70, 300])
@pytest.mark.parametrize("score", [mx.MX_ROUTE_SOFTMAX, mx.MX_ROUTE_SIGMOID])
@pytest.mark.parametrize("bias", [False, True])
def test_route_logits_below_the_range_of_fp32_scores(E, score, bias):
    """exp(-l) overflows FP32 at l = -88.7 and FP64 at -709.8: between them the weights are the scores' ratios all the
    same, with a bias of zeros or none."""
    rows = [[-95, -96, -97, -98], [-85, -92, -92.5, -103], [-88, -88.5, -88.75, -89], [-64, -64.25, -63.75, -65],
            [-100, -110, -120, -130], [-650, -651, -652.5, -690], [-700, -720, -800, -900], [3, -20, -70, -140],
            [-90, -np.inf, -np.inf, -91], [-720, -721, -722, -723]]
    l = np.full((len(rows), E), -1000.0, dtype=np.float32)
    for t, r in enumerate(rows):
        l[t, [5, E - 3, 17, 40]] = r
    b = np.zeros(E, dtype=np.float32) if bias else None
    say("route far logits", E, score, bias)
    for k in (3, 4):
        _check_route(l.astype(np.float64), _f32(l), k, b, score, True, 2.5)
        # scores as they are, to FP32's smallest steps (2^-149)
        got = mx.mx_moe_route(_f32(l), k, bias=None if b is None else _f32(b), score=score, renormalize=False)[1]
        ref = M.route(l.astype(np.float64), k, b, score, False)[1]
        assert np.all(np.abs(got.cpu().numpy() - ref) <= 2.0 ** -17 * ref + 2.0 ** -149)


@pytest.mark.parametrize("E", [16, 300])
@pytest.mark.parametrize("score", [mx.MX_ROUTE_SOFTMAX, mx.MX_ROUTE_SIGMOID])
def test_route_bias_of_the_lowest_value_beside_masked_experts(E, score):
    """A bias of the type's lowest value ranks its expert behind all others with a finite key, but before the masked."""
    low = np.finfo(np.float32).min
    l = np.full((4, E), -np.inf, dtype=np.float32)
    l[0, [3, 9]] = 1.0, 2.0                    # two left, the second behind the lowest bias
    l[1, [3, 9, 11]] = 1.0, 2.0, 0.5
    l[2, 9] = 2.0
    l[3] = 0.25
    say("route lowest bias", E, score)
    for bias in (low, np.float32(-3.4e38), np.float32(low * 0.999)):
        b = np.zeros(E, dtype=np.float32)
        b[9] = bias
        for k in (1, 2, 3):
            _check_route(l.astype(np.float64), _f32(l), k, b, score)


# ---------------------------------------------------------------- products

def _weights(rng, lead, N, K, fmt):
    w = workloads.weight_codes(rng, lead + (N, K))
    if fmt == "mx":
        return w, workloads.scale_bytes(rng, lead + (N, K // 32), -10, -4)
    return w, (1e-3 * (0.5 + rng.random(lead + (-(-N // 128), -(-K // 128))))).astype(np.float32)


def _scale_dev(ws):
    return dev_u8(ws) if ws.dtype == np.uint8 else _f32(ws)


def _close(got_bits, ref, extra=None, what=""):
    """helpers.assert_gemm_close with an addition to the bound; NaN rows of ref must be NaN."""
    g = F.bf16_to_f64(got_bits)
    nan = np.isnan(ref)
    assert np.array_equal(np.isnan(g), nan), f"{what}: NaN in other places"
    if nan.all():
        return
    rms = np.sqrt(np.mean(ref[~nan] ** 2))
    bound = 2.0 ** -7 * np.abs(ref) + 1e-3 * rms + (0 if extra is None else extra)
    err = np.abs(g - ref)
    bad = ~nan & ~(err <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {ref.size} outside, first at {np.argwhere(bad)[0]}"


def _swiglu_extra(x_bits, w, ws, offsets, slots=None, k=1):
    """|Q(h-) - Q(h+)| @ |W|^T, h-+ the BF16 roundings of silu(gate) * up moved by its FP32 evaluation's error, below
    2^-16 relative: the exponent's rounding moves the exponential by |gate| 2^-24 <= 2^-17 (|gate| <= 128: beyond, the
    result is 0 or gate * up), and the exponential, an addition, a reciprocal and two products by at most 8 steps of
    2^-24."""
    h = M.swiglu(x_bits)
    if slots is not None:
        h = h[slots // k]
    lo, hi = F.f64_to_bf16_rne(h * (1 - 2.0 ** -16)), F.f64_to_bf16_rne(h * (1 + 2.0 ** -16))
    out = np.zeros((h.shape[0], w.shape[1]))
    for e in range(w.shape[0]):
        s = slice(offsets[e], offsets[e + 1])
        if offsets[e + 1] > offsets[e]:
            a, wv = M.operands(lo[s], w[e], ws[e])
            b, _ = M.operands(hi[s], w[e], ws[e])
            out[s] = np.nan_to_num(np.abs(a - b)) @ np.abs(wv).T
    return out


def _sizes(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def _run_grouped(seed, fmt, counts, N, K, act=False, gather=None, k=1, spoil=None):
    rng = np.random.default_rng(seed)
    E, off = len(counts), _sizes(counts)
    S = int(off[-1])
    rows = S if gather is None else gather
    x = workloads.activations(rng, rows, 2 * K if act else K)
    w, ws = _weights(rng, (E,), N, K, fmt)
    slots = None if gather is None else rng.integers(0, rows * k, S).astype(np.int32)
    if spoil:
        spoil(x, w, ws, slots)
    say("grouped", fmt, "S", S, "E", E, "N", N, "K", K, "act", act, "gather", gather)
    out = mx.mx_grouped_linear(dev_u16(x), dev_u8(w), _scale_dev(ws), _i32(off),
                               row_slot=None if slots is None else _i32(slots), k=k,
                               act=mx.MX_ACT_SWIGLU if act else mx.MX_ACT_NONE)
    torch.cuda.synchronize()
    ref = M.grouped_linear(x, w, ws, off, slots, k, act)
    extra = _swiglu_extra(x, w, ws, off, slots, k) if act else None
    _close(host_u16(out), ref, extra, f"{fmt} {counts} N={N} K={K}")
    return out


MX_K = [32, 96, 128, 160, 288, 576, 1152, 2304]
F32_K = [16, 112, 128, 144, 272, 1040, 2304]


@pytest.mark.parametrize("fmt,K", [("mx", k) for k in MX_K] + [("f32", k) for k in F32_K])
@pytest.mark.parametrize("counts,N", [([1], 16), ([3, 0, 1, 33], 80), ([0, 0, 70], 144), ([100, 1, 0, 90], 272)])
def test_grouped_small(fmt, K, counts, N):
    """Tiles of 32 and 64 rows: every K tail, empty experts, edges in N."""
    _run_grouped(K + N, fmt, counts, N, K)


@pytest.mark.parametrize("fmt", ["mx", "f32"])
@pytest.mark.parametrize("counts,N", [([2600], 6656), ([2343, 7], 6944), ([0, 2560, 0], 9472)])
def test_grouped_last_round(fmt, counts, N):
    """Counts of 256-row tiles a little, a quarter and a half above what the compute units hold at once."""
    _run_grouped(N, fmt, counts, N, 160 if fmt == "mx" else 272)


@pytest.mark.parametrize("fmt,K", [("mx", 160), ("mx", 512), ("mx", 1056), ("mx", 1184), ("mx", 1280), ("f32", 144), ("f32", 640)])
@pytest.mark.parametrize("act", [False, True])
@pytest.mark.parametrize("counts,N", [([129, 300, 0, 131, 128], 4112), ([1025, 40, 257, 256], 4400), ([2600], 7696),
                                      ([700, 0, 1300, 257], 8208)])
def test_grouped_large_tiles(fmt, K, act, counts, N):
    """Tiles of 128 and 256 rows, ragged in both directions."""
    _run_grouped(7 * K + N, fmt, counts, N, K, act=act)


@pytest.mark.parametrize("fmt,K", [("mx", 32), ("mx", 160), ("mx", 288), ("mx", 1152), ("f32", 16), ("f32", 144), ("f32", 272),
                                   ("f32", 1040)])
@pytest.mark.parametrize("counts,N", [([60, 100, 0, 90], 4112), ([150, 200, 170], 4112), ([700], 4112), ([250], 5136)])
def test_grouped_waves_split_over_k(fmt, K, counts, N):
    """Tiles of 64 x 128 and 128 x 128, fewer than compute units: every K tail, K of one stage among them."""
    _run_grouped(5 * K + N, fmt, counts, N, K)


@pytest.mark.parametrize("K", [1056, 1184, 1280])
@pytest.mark.parametrize("act,gather", [(False, None), (True, None), (False, 900), (True, 900)])
def test_grouped_large_groups(K, act, gather):
    """Groups of a thousand rows and more on average, some empty or small, from x or gathered from fewer rows of it."""
    _run_grouped(K, "mx", [1300, 0, 2700, 257], 4112, K, act=act, gather=gather, k=3)


@pytest.mark.parametrize("fmt", ["mx", "f32"])
@pytest.mark.parametrize("counts,N,K", [([4, 0, 2], 80, 288), ([40, 90], 144, 160), ([150, 100], 8208, 160), ([700, 500], 5136, 160)])
def test_grouped_gathers_gate_and_up(fmt, counts, N, K):
    """SwiGLU of gathered rows, for each size of tile."""
    _run_grouped(N + K, fmt, counts, N, K, act=True, gather=37, k=2)


@pytest.mark.parametrize("fmt", ["mx", "f32"])
@pytest.mark.parametrize("T,E,k,N,K", [(1, 8, 2, 64, 288), (5, 16, 4, 80, 1152), (61, 4, 3, 272, 576), (700, 3, 2, 1040, 320)])
def test_grouped_gathers_router_slots(fmt, T, E, k, N, K):
    rng = np.random.default_rng(T)
    x = workloads.activations(rng, T, K)
    w, ws = _weights(rng, (E,), N, K, fmt)
    l = rng.standard_normal((T, E)).astype(np.float32)
    say("grouped gather", fmt, T, E, k)
    _, _, off, rs, _ = mx.mx_moe_route(_f32(l), k)
    out = mx.mx_grouped_linear(dev_u16(x), dev_u8(w), _scale_dev(ws), off, row_slot=rs, k=k)
    torch.cuda.synchronize()
    _close(host_u16(out), M.grouped_linear(x, w, ws, off.cpu().numpy(), rs.cpu().numpy(), k))


@pytest.mark.parametrize("fmt,K", [("mx", 288), ("mx", 384), ("f32", 272), ("f32", 384)])
@pytest.mark.parametrize("counts,N", [([5, 0, 31, 9], 8208), ([60, 3, 64, 0, 40], 8208), ([100, 128, 70], 8208),
                                      ([1] * 64, 2320), ([200, 10, 90, 0, 300, 65], 5136)])
def test_grouped_shares_of_many_columns(fmt, K, counts, N):
    """Enough columns that a workgroup's share holds several tiles, begins inside a block of 128 columns and ends in
    another expert's, with groups of several row tiles."""
    _run_grouped(3 * K + N, fmt, counts, N, K)


@pytest.mark.parametrize("fmt,K", [("mx", 1184), ("mx", 1280), ("f32", 1168), ("f32", 1280)])
@pytest.mark.parametrize("counts,N,gather", [([5, 0, 31, 9], 8208, None), ([1] * 64, 2320, None), ([40, 0, 20, 3], 4112, 7),
                                             ([0, 32, 1, 33, 0, 2], 5136, 50)])
def test_grouped_shares_of_long_rows(fmt, K, counts, N, gather):
    """The same for rows of more stages, which small groups take there."""
    _run_grouped(2 * K + N, fmt, counts, N, K, gather=gather, k=2)


def _list_bytes(BM, S, E):
    """Bytes of the list of row tiles of BM rows in the workspace of a grouped product."""
    return -(-32 * (1 + S // BM + min(S, E)) // 256) * 256


@pytest.mark.parametrize("fmt,K", [("mx", 32), ("mx", 96), ("mx", 288), ("mx", 512), ("mx", 576), ("mx", 1024), ("f32", 16),
                                   ("f32", 112), ("f32", 272), ("f32", 512), ("f32", 640), ("f32", 1024)])
@pytest.mark.parametrize("counts", [[249, 1, 1, 1, 1, 1, 1, 1], [140, 70, 20, 20, 3, 2, 0, 1]])
@pytest.mark.parametrize("gather,act", [(None, False), (37, False), (37, True)])
def test_grouped_skewed_groups_of_short_rows(fmt, K, counts, gather, act):
    """Small groups on average, one of them large: 32-row tiles, of which a workgroup's share holds two or three, each of
    one or two super-stages of 512 K.  Some gathered rows have no source."""
    N, E, S = 2048, len(counts), sum(counts)
    rows = S if gather is None else gather
    rest = sum(-(-b // 256) * 256 for b in (rows * -(-K // 128) * 128, rows * -(-K // 512) * 16))
    assert mx.mx_grouped_linear_workspace_bytes(rows, S, E, N, K) - rest == _list_bytes(32, S, E) != _list_bytes(128, S, E)

    def spoil(x, w, ws, slots):
        slots[[0, 131, 250]] = [-1, 37 * 2, 2 ** 31 - 1]
    _run_grouped(K + counts[0], fmt, counts, N, K, act=act, gather=gather, k=2, spoil=spoil if gather and not act else None)


@pytest.mark.parametrize("fmt", ["mx", "f32"])
def test_grouped_bad_slots_and_nonfinite_inputs(fmt):
    def spoil(x, w, ws, slots):
        slots[[0, 50, 199]] = [-1, 37 * 2, 2 ** 31 - 1]    # outside x: 37 rows of k = 2 slots
        slots[5] = slots[6]                                # the same row twice
        x[3, 7], x[4, 100], x[5, :] = 0x7F80, 0x7FC0, 0    # Inf, NaN, a row of zeros
    _run_grouped(3, fmt, [40, 160, 0, 60], 144, 160, gather=37, k=2, spoil=spoil)
    _run_grouped(4, fmt, [400, 600, 0, 260], 4112, 160, gather=37, k=2, spoil=spoil)


@pytest.mark.parametrize("fmt", ["mx", "f32"])
def test_grouped_extreme_magnitudes(fmt):
    """Activation blocks at the ends of BF16: subnormals, the largest finite values, and tiny next to huge blocks."""
    rng = np.random.default_rng(8)
    K, N = 256, 32
    x = rng.standard_normal((12, K)).astype(np.float32)
    x[0] *= 1e-38
    x[1] *= 1e-30
    x[2, :128] *= 1e-20
    x[3] *= 1e20
    bits = workloads.to_bf16_bits(x)
    bits[4, 9] = 0x7F7F                                    # the largest finite BF16
    bits[5] = 1                                            # the smallest subnormal
    bits[6] = 0x8000
    w = workloads.weight_codes(rng, (1, N, K))
    ws = np.full((1, N, K // 32), 127 - 40, np.uint8) if fmt == "mx" else np.full((1, 1, 2), 2.0 ** -40, np.float32)
    say("grouped extremes", fmt)
    out = mx.mx_grouped_linear(dev_u16(bits), dev_u8(w), _scale_dev(ws), _i32([0, 12]))
    torch.cuda.synchronize()
    ref = M.grouped_linear(bits, w, ws, [0, 12])
    for r in range(12):                                    # each row by its own magnitude
        _close(host_u16(out)[r:r + 1], np.where(np.abs(ref[r:r + 1]) < 2.0 ** -126, 0, ref[r:r + 1]), 2.0 ** -126, f"row {r}")


def test_grouped_nan_weight_and_scale_stay_in_their_column():
    def spoil(x, w, ws, slots):
        w[1, 3, 70] = 0x7F
        ws[1, 9, 4] = 0xFF
        w[0, 15, 159] = 0xFF                               # in the last chunk, which K's tail reads again
    _run_grouped(11, "mx", [20, 20], 32, 160, spoil=spoil)


def test_grouped_leaves_other_rows():
    """Rows behind the last expert and before the first keep what they held; offsets past S are cut."""
    rng = np.random.default_rng(9)
    x = workloads.activations(rng, 300, 96)
    w, ws = _weights(rng, (3,), 48, 96, "mx")
    say("grouped offsets")
    for off, lo, hi in (([10, 40, 40, 170], 10, 170), ([0, 5, 290, 900], 0, 300), ([0, 0, 0, 0], 0, 0),
                        ([-4, 2, 2, 50], 0, 50)):
        out = torch.full((300, 48), 7.0, dtype=torch.bfloat16, device="cuda")
        mx.mx_grouped_linear(dev_u16(x), dev_u8(w), dev_u8(ws), _i32(off), out=out)
        torch.cuda.synchronize()
        ref = M.grouped_linear(x, w, ws, np.clip(off, 0, 300))
        ref[:lo], ref[hi:] = 7.0, 7.0
        _close(host_u16(out), ref, what=str(off))
        assert (out[:lo] == 7).all() and (out[hi:] == 7).all()


def test_grouped_many_experts():
    rng = np.random.default_rng(12)
    counts = rng.integers(0, 4, 700)
    _run_grouped(12, "mx", counts.tolist(), 16, 64)


@pytest.mark.parametrize("fmt", ["mx", "f32"])
def test_grouped_equal_tokens_are_equal(fmt):
    """One x row for every row of a large group: whatever tile and lane a row falls on, its outputs are the same."""
    rng = np.random.default_rng(13)
    x = workloads.activations(rng, 1, 640)
    w, ws = _weights(rng, (1,), 528, 640, fmt)
    for S in (7, 60, 1000, 9000):
        out = mx.mx_grouped_linear(dev_u16(x), dev_u8(w), _scale_dev(ws), _i32([0, S]), row_slot=_i32(np.zeros(S)))
        assert (out == out[0]).all()


@pytest.mark.parametrize("fmt", ["mx", "f32"])
@pytest.mark.parametrize("counts,N,K", [([1, 0, 3], 4112, 2304), ([40, 90], 144, 160), ([150, 100], 8208, 160),
                                        ([700, 500], 5136, 1152), ([1300, 0, 2700, 257], 4112, 1280)])
def test_grouped_repeats_bit_for_bit(fmt, counts, N, K):
    """Equal calls give equal bits, for each kind of tile."""
    rng = np.random.default_rng(N + K)
    off = _sizes(counts)
    x = dev_u16(workloads.activations(rng, int(off[-1]), K))
    w, ws = _weights(rng, (len(counts),), N, K, fmt)
    w, ws, off = dev_u8(w), _scale_dev(ws), _i32(off)
    say("grouped repeats", fmt, counts, N, K)
    first = mx.mx_grouped_linear(x, w, ws, off)
    for _ in range(5):
        assert torch.equal(mx.mx_grouped_linear(x, w, ws, off).view(torch.int16), first.view(torch.int16))


# ---------------------------------------------------------------- block 128

@pytest.mark.parametrize("Mr,N,K", [(1, 16, 16), (1, 5120, 2304), (2, 144, 144), (17, 272, 1040), (33, 1024, 4096),
                                    (64, 4096, 576), (65, 80, 2304), (129, 1040, 4112), (30, 16400, 144), (100, 16400, 272), (513, 2064, 272),
                                    (2100, 2320, 272), (4200, 5136, 144)])
def test_block128(Mr, N, K):
    rng = np.random.default_rng(Mr + N + K)
    x = workloads.activations(rng, Mr, K)
    w, ws = _weights(rng, (), N, K, "f32")
    say("block128", Mr, N, K)
    out = mx.mx_linear_block128(dev_u16(x), dev_u8(w), _f32(ws))
    torch.cuda.synchronize()
    _close(host_u16(out), M.linear_block128(x, w, ws))


def test_block128_scales_that_are_no_powers_of_two():
    """Signs and magnitudes of the block scales reach the output as they are."""
    rng = np.random.default_rng(2)
    x = workloads.activations(rng, 40, 384)
    w, _ = _weights(rng, (), 256, 384, "f32")
    ws = np.array([[1 / 3, -2.7, 1e-4], [0.0, 5e3, np.pi]], dtype=np.float32)
    out = mx.mx_linear_block128(dev_u16(x), dev_u8(w), _f32(ws))
    torch.cuda.synchronize()
    ref = M.linear_block128(x, w, ws)
    _close(host_u16(out)[:, :128], ref[:, :128])
    _close(host_u16(out)[:, 128:], ref[:, 128:])


# --------------------------------------------------------------------- join

@pytest.mark.parametrize("T,k,N", [(1, 1, 8), (1, 8, 5120), (5, 3, 16), (64, 6, 1032), (1000, 8, 2304), (3, 40, 264),
                                   (7, 2, 40), (9, 4, 520), (6, 5, 264), (4, 7, 1032), (5, 9, 264), (3, 12, 72), (3, 17, 8)])
@pytest.mark.parametrize("shared", [False, True])
def test_combine(T, k, N, shared):
    rng = np.random.default_rng(T + k + N)
    y = workloads.activations(rng, T * k, N)
    sr = rng.permutation(T * k).astype(np.int32).reshape(T, k)
    wt = rng.random((T, k)).astype(np.float32)
    sh = workloads.activations(rng, T, N) if shared else None
    if T > 1:
        sr[0, 0], sr[1, -1], wt[1, 0] = -1, T * k, 0.0     # dropped slots
        y[sr[1, 0]] = 0x7FC0                               # NaN behind a weight of 0
        sr[2] = sr[2, 0]                                   # one row for every slot
    say("combine", T, k, N, shared)
    out = mx.mx_moe_combine(dev_u16(y), _i32(sr), _f32(wt), shared=None if sh is None else dev_u16(sh))
    torch.cuda.synchronize()
    ref = M.combine(y, sr, wt, sh)
    size = M.combine(y & 0x7FFF, sr, np.abs(wt), None if sh is None else sh & 0x7FFF)
    got = F.bf16_to_f64(host_u16(out))
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + (k + 2) * 2.0 ** -23 * size)
    if shared:
        buf = dev_u16(sh)
        mx.mx_moe_combine(dev_u16(y), _i32(sr), _f32(wt), shared=buf, out=buf)
        assert torch.equal(buf.view(torch.int16), out.view(torch.int16))


# ----------------------------------------------------------------- together

def _layer(rng, E, hidden, inner, fmt):
    up, ups = _weights(rng, (E,), 2 * inner, hidden, fmt)
    down, downs = _weights(rng, (E,), hidden, inner, fmt)
    # near-unit activations: weights of random codes are large
    ups = ups - 4 if ups.dtype == np.uint8 else ups * np.float32(2.0 ** -4)
    return up, ups, down, downs


def _run_layer(x, logits, bias, k, dev, shared):
    ids, wt, off, rs, sr = mx.mx_moe_route(logits, k, bias=bias, score=mx.MX_ROUTE_SIGMOID, scale=2.5)
    h = mx.mx_grouped_linear(x, dev[0], dev[1], off, row_slot=rs, k=k)
    y = mx.mx_grouped_linear(h, dev[2], dev[3], off, act=mx.MX_ACT_SWIGLU)
    return mx.mx_moe_combine(y, sr, wt, shared=shared), (ids, wt, off, rs, sr, h, y)


@pytest.mark.parametrize("fmt", ["mx", "f32"])
@pytest.mark.parametrize("T,E,k,hidden,inner", [(1, 8, 2, 256, 288), (70, 16, 4, 512, 160), (900, 5, 2, 640, 544)])
def test_layer_stage_by_stage(fmt, T, E, k, hidden, inner):
    """A whole layer, each stage against the oracle on the stage's own input."""
    rng = np.random.default_rng(T + E)
    x, sh = workloads.activations(rng, T, hidden), workloads.activations(rng, T, hidden)
    l, b = rng.standard_normal((T, E)).astype(np.float32), (0.1 * rng.standard_normal(E)).astype(np.float32)
    up, ups, down, downs = _layer(rng, E, hidden, inner, fmt)
    dev = [dev_u8(up), _scale_dev(ups), dev_u8(down), _scale_dev(downs)]
    say("layer", fmt, T, E, k)
    out, (ids, wt, off, rs, sr, h, y) = _run_layer(dev_u16(x), _f32(l), _f32(b), k, dev, dev_u16(sh))
    torch.cuda.synchronize()
    rid, rw, roff, rrs, rsr = M.route(l.astype(np.float64), k, b, M.SIGMOID, True, 2.5)
    assert np.array_equal(ids.cpu().numpy(), rid) and np.array_equal(off.cpu().numpy(), roff)
    _close(host_u16(h), M.grouped_linear(x, up, ups, roff, rrs, k))
    hb = host_u16(h)
    _close(host_u16(y), M.grouped_linear(hb, down, downs, roff, act=True), _swiglu_extra(hb, down, downs, roff))
    ref = M.combine(host_u16(y), rsr, wt.cpu().numpy(), sh)
    got = F.bf16_to_f64(host_u16(out))
    size = M.combine(host_u16(y) & 0x7FFF, rsr, wt.cpu().numpy(), sh & 0x7FFF)
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + (k + 2) * 2.0 ** -23 * size)


@pytest.mark.parametrize("fmt", ["mx", "f32"])
def test_layer_in_a_graph(fmt):
    """Captured once, replayed with new inputs between eager calls on the same buffers: equal bits each time."""
    rng = np.random.default_rng(21)
    T, E, k, hidden, inner = 150, 12, 3, 384, 160
    up, ups, down, downs = _layer(rng, E, hidden, inner, fmt)
    dev = [dev_u8(up), _scale_dev(ups), dev_u8(down), _scale_dev(downs)]
    x = torch.zeros((T, hidden), dtype=torch.bfloat16, device="cuda")
    l = torch.zeros((T, E), device="cuda")
    b = torch.zeros(E, device="cuda")
    say("layer graph", fmt)
    _run_layer(x, l, b, k, dev, None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, _ = _run_layer(x, l, b, k, dev, None)
    gen = torch.Generator(device="cuda").manual_seed(3)
    for _ in range(4):
        x.copy_(torch.randn((T, hidden), generator=gen, device="cuda"))
        l.copy_(torch.randn((T, E), generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        eager, _ = _run_layer(x, l, b, k, dev, None)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)


def test_layer_on_two_streams():
    """Two calls at once on their own streams and workspaces give what one after the other gives."""
    rng = np.random.default_rng(31)
    T, E, k, hidden, inner = 600, 8, 2, 512, 288
    up, ups, down, downs = _layer(rng, E, hidden, inner, "mx")
    dev = [dev_u8(up), _scale_dev(ups), dev_u8(down), _scale_dev(downs)]
    ins = [(dev_u16(workloads.activations(rng, T, hidden)), _f32(rng.standard_normal((T, E)))) for _ in range(2)]
    want = [_run_layer(x, l, None, k, dev, None)[0] for x, l in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = []
        for s, (x, l) in zip(streams, ins):
            with torch.cuda.stream(s):
                got.append(_run_layer(x, l, None, k, dev, None)[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("fmt", ["mx", "f32"])
@pytest.mark.parametrize("rows", [3, 300, 600])
def test_grouped_weight_behind_4_gb(fmt, rows):
    """The last expert's weight lies behind 2^32 bytes: its last columns equal those of an expert of their own, for 32-,
    128- and 256-row tiles.  x is 0 or +-448 (one power of two as its scale, or 1), the codes are +-1 and +-2 and the
    weight's scales powers of two within 2^3 of each other: every sum is an integer below 448 * 2^20 in steps of 448, exact
    in any order."""
    E, N, K = 3, 65552, 23040
    say("grouped behind 4 GB", fmt, rows)
    gen = torch.Generator(device="cuda").manual_seed(rows)
    w = torch.randint(0, 4, (E, N, K), generator=gen, dtype=torch.uint8, device="cuda")
    w = (w & 1).mul_(8).add_(0x38).bitwise_or_((w & 2).mul_(64))
    if fmt == "mx":
        ws = torch.randint(124, 128, (E, N, K // 32), generator=gen, dtype=torch.uint8, device="cuda")
    else:
        ws = 2.0 ** torch.randint(-3, 1, (E, -(-N // 128), K // 128), generator=gen, device="cuda").float()
    x = (448 * torch.randint(-1, 2, (rows, K), generator=gen, device="cuda")).bfloat16()
    out = mx.mx_grouped_linear(x, w, ws, _i32([0, 0, 0, rows]))
    n0 = N - 272
    part = mx.mx_grouped_linear(x, w[2, n0:].contiguous()[None], ws[2:, n0 if fmt == "mx" else n0 // 128:].contiguous(),
                                _i32([0, rows]))
    torch.cuda.synchronize()
    assert part.abs().max() > 0 and torch.equal(out[:, n0:], part)


def test_combine_behind_4_gb():
    """Rows of y and out behind 2^32 bytes and 2^31 elements."""
    T, N = 70001, 32768
    say("combine behind 4 GB")
    y = torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
    y.copy_((torch.arange(T, device="cuda") % 251).bfloat16()[:, None].expand(T, N))
    row = torch.arange(T, dtype=torch.int32, device="cuda").flip(0)[:, None].contiguous()
    out = mx.mx_moe_combine(y, row, torch.full((T, 1), 2.0, device="cuda"))
    torch.cuda.synchronize()
    for t in (0, 1, 32767, 32768, 65535, 65536, T - 1):
        assert (out[t] == 2 * ((T - 1 - t) % 251)).all(), t


def test_launch_counters():
    mx.mx_reset_counters()
    off = _i32([0, 4])
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((1, 16, 64), dtype=torch.uint8, device="cuda")
    mx.mx_grouped_linear(x, w, torch.full((1, 16, 2), 127, dtype=torch.uint8, device="cuda"), off)
    mx.mx_linear_block128(x, w[0], torch.ones((1, 1), device="cuda"))
    mx.mx_moe_route(torch.zeros((4, 4), device="cuda"), 1)
    mx.mx_moe_combine(x, torch.zeros((4, 1), dtype=torch.int32, device="cuda"), torch.ones((4, 1), device="cuda"))
    torch.cuda.synchronize()
    c = mx.mx_get_counters()
    assert {n: v for n, v in c.items() if v} == {"grouped_linear": 1, "linear_block128": 1, "moe_route": 1,
                                                 "moe_combine": 1}
