"""Pins of the mixture-of-experts oracle: hand cases, brute-force loops, and the formulas at their edges."""

import math

import numpy as np
import pytest

import workloads
from oracle import formats as F
from oracle import gemm as G
from oracle import moe as M


def test_route_hand_case():
    # token 0: experts 2 and 0 (logits 3 > 1); token 1: a tie of 1 and 3 goes to the lower index first
    l = np.array([[1.0, 0.0, 3.0, -1.0], [0.0, 2.0, 1.0, 2.0]])
    ids, w, off, row_slot, slot_row = M.route(l, 2)
    assert ids.tolist() == [[2, 0], [1, 3]]
    a = 1 / (1 + math.exp(-2.0))                     # e^3 / (e^3 + e^1)
    assert np.allclose(w, [[a, 1 - a], [0.5, 0.5]], rtol=1e-15)
    # slots 0..3 hold experts 2, 0, 1, 3
    assert off.tolist() == [0, 1, 2, 3, 4]
    assert row_slot.tolist() == [1, 2, 0, 3]
    assert slot_row.tolist() == [[2, 0], [1, 3]]


def test_route_bias_picks_but_does_not_weigh():
    l = np.array([[0.0, 1.0, 2.0]])
    ids, w, *_ = M.route(l, 1, bias=[5.0, 0.0, 0.0], score=M.SIGMOID, renormalize=False, scale=2.0)
    assert ids.tolist() == [[0]] and w[0, 0] == 1.0   # sigmoid(0) * 2


def test_route_masks_and_nan():
    inf = np.inf
    ids, w, *_ = M.route(np.array([[-inf, 1.0, np.nan, -inf], [-inf] * 4, [inf, 0.0, 0.0, 0.0]]), 2)
    assert ids[0].tolist() == [1, 0] and w[0].tolist() == [1.0, 0.0]
    assert ids[1].tolist() == [0, 1] and w[1].tolist() == [0.0, 0.0]
    assert ids[2].tolist() == [0, 1] and w[2].tolist() == [1.0, 0.0]


def test_group_is_a_stable_sort():
    rng = np.random.default_rng(0)
    ids = rng.integers(0, 7, (50, 3))
    off, row_slot, slot_row = M.group(ids, 9)
    assert np.array_equal(row_slot, np.argsort(ids.reshape(-1), kind="stable"))
    assert np.array_equal(slot_row.reshape(-1)[row_slot], np.arange(150))
    assert off[-1] == 150 and off[7] == 150


def test_quantise_f32_hand_case():
    # amax 2 -> scale 2/448; 1 -> 224 exactly; 0.3 -> about 67, grid spacing 8 between 64 and 128: 64
    x = np.zeros((1, 200), dtype=np.float32)
    x[0, :3] = [2.0, 1.0, -0.30078125]               # 0.30078125 is a BF16; * 224 = 67.375 -> 64
    x[0, 130] = 7.0                                  # the second, short block has its own scale
    q = M.quantise_f32(workloads.to_bf16_bits(x))
    s = float(np.float32(2.0 / 448.0))
    assert q[0, :4].tolist() == [448 * s, 224 * s, -64 * s, 0.0]
    assert q[0, 130] == 448 * float(np.float32(7.0 / 448.0))


def test_quantise_f32_breaks_ties_to_even():
    # amax 448: codes are x itself; 17 lies between 16 and 18 (spacing 2) -> 16, 19 -> 20
    x = np.array([[448.0, 17.0, 19.0, -17.0]], dtype=np.float32)
    q = M.quantise_f32(workloads.to_bf16_bits(np.pad(x, ((0, 0), (0, 12)))))
    assert q[0, :4].tolist() == [448.0, 16.0, 20.0, -16.0]


def test_quantise_f32_nonfinite_and_zero_blocks():
    x = np.zeros((2, 256), dtype=np.float32)
    x[0, 5], x[1, 200] = np.inf, 1.0
    q = M.quantise_f32(workloads.to_bf16_bits(x))
    assert np.isnan(q[0, :128]).all() and (q[0, 128:] == 0).all()
    assert (q[1, :128] == 0).all() and q[1, 200] == 448 * float(np.float32(1 / 448))


def test_weight_f32_blocks_by_loops():
    rng = np.random.default_rng(1)
    w = workloads.weight_codes(rng, (144, 272))
    s = rng.random((2, 3)).astype(np.float32)
    v = M.weight_f32(w, s)
    for n, k in ((0, 0), (127, 127), (128, 128), (143, 271), (5, 256)):
        assert v[n, k] == F.e4m3_decode(w[n, k], F.OCP) * float(s[n // 128, k // 128])


@pytest.mark.parametrize("fmt", ["mx", "f32"])
def test_grouped_linear_by_loops(fmt):
    rng = np.random.default_rng(2)
    E, N, K, T, k = 4, 16, 64, 5, 2
    x = workloads.activations(rng, T, K)
    w = workloads.weight_codes(rng, (E, N, K))
    ws = (workloads.scale_bytes(rng, (E, N, K // 32), -6, -2) if fmt == "mx"
          else rng.random((E, 1, 1)).astype(np.float32))
    ids = np.array([[3, 0], [0, 1], [3, 1], [0, 3], [1, 0]])
    off, row_slot, _ = M.group(ids, E)
    out = M.grouped_linear(x, w, ws, off, row_slot, k)
    xq = M.quantise_mx(x) if fmt == "mx" else M.quantise_f32(x)
    for r, s in enumerate(row_slot):
        e = ids[s // k, s % k]
        wv = G.scaled_operand(w[e], ws[e], 32) if fmt == "mx" else M.weight_f32(w[e], ws[e])
        for n in range(N):
            assert math.isclose(out[r, n], math.fsum(xq[s // k, i] * wv[n, i] for i in range(K)), rel_tol=1e-12,
                                abs_tol=1e-12)


def test_swiglu_points():
    x = workloads.to_bf16_bits(np.array([[0.0, 1.0, -200.0, 50.0, 2.0, 3.0, 4.0, -1.0]], dtype=np.float32))
    h = M.swiglu(x)[0]
    assert h[0] == 0.0 and math.isclose(h[1], 3.0 / (1 + math.exp(-1.0))) and abs(h[2]) < 1e-80 and h[3] == -50.0


def test_combine_drops_slots():
    y = workloads.to_bf16_bits(np.array([[1.0, 2.0], [np.nan, np.inf]], dtype=np.float32))
    out = M.combine(y, np.array([[0, 1], [-1, 0]]), np.array([[0.5, 0.0], [1.0, 2.0]], dtype=np.float32))
    assert out.tolist() == [[0.5, 1.0], [2.0, 4.0]]
