"""Pins of oracle/attn.py: hand cases and loops over the definition."""

import math

import numpy as np

import workloads
from oracle import attn as A
from oracle import formats as F


def test_two_keys_by_hand():
    # scores 0 and ln 3: weights 1/4 and 3/4
    q = np.array([[[1.0, 0.0]]])
    k = np.array([[[0.0, 5.0]], [[math.log(3.0), 0.0]]])
    v = np.array([[[4.0, -4.0]], [[8.0, 0.0]]])
    out, size, spread = A.attend(q, k, v, 1.0)
    assert np.allclose(out, [[[7.0, -1.0]]]) and np.allclose(size, [[[7.0, 1.0]]])
    assert np.allclose(spread, math.log(3.0))


def test_rows_without_keys_are_zero_and_the_rest_is_aligned_to_the_end():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((4, 2, 8)), rng.standard_normal((2, 1, 8)), rng.standard_normal((2, 1, 8))
    out, _, _ = A.attend(q, k, v, 0.3)
    assert not out[:2].any()
    assert np.allclose(out[2], v[0])                       # the third row sees one key
    s = 0.3 * q[3] @ k[:, 0].T
    w = np.exp(s) / np.exp(s).sum(1, keepdims=True)
    assert np.allclose(out[3], w @ v[:, 0])


def test_groups_share_a_key_head():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 6, 4)), rng.standard_normal((5, 2, 4)), rng.standard_normal((5, 2, 4))
    out, _, _ = A.attend(q, k, v, 1.0)
    for h in range(6):
        for i in range(3):
            n = 5 - 3 + i + 1
            w = [math.exp(float(q[i, h] @ k[j, h // 3])) for j in range(n)]
            want = sum(w[j] * v[j, h // 3] for j in range(n)) / sum(w)
            assert np.allclose(out[i, h], want)


def test_write_and_sequence_round_trip():
    rng = np.random.default_rng(2)
    pages, heads, page, D, T = 4, 2, 16, 64, 20
    x = workloads.activations(rng, T, heads * D).reshape(T, heads, D)
    slots = rng.permutation(pages * page)[:T]
    bf, none = A.write(x, slots, np.zeros((pages, heads, page, D), np.uint16), None)
    assert none is None
    c, s = A.write(x, slots, np.zeros((pages, heads, page, D), np.uint8), np.zeros((pages, heads, page, 2), np.uint8))
    for t in range(T):
        p, i = divmod(int(slots[t]), page)
        assert np.array_equal(bf[p, :, i], x[t])
        got = A.values(c[p, :, i], s[p, :, i])
        want = F.bf16_to_f64(x[t])
        amax = np.abs(want).reshape(heads, 2, 32).max(2).repeat(32, 1).reshape(heads, D)
        # a code is within half a step: 2^-4 of its value, or of the smallest normal 2^-6 under a scale of at most 2 amax / 448
        assert np.all(np.abs(got - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * 2 * amax / 448))
    table = [2, 0, 9]
    seq = A.sequence(c, s, table, 37)
    assert np.array_equal(seq[:16], A.values(c[2], s[2]).transpose(1, 0, 2))
    assert np.array_equal(seq[16:32], A.values(c[0], s[0]).transpose(1, 0, 2))
    assert np.isnan(seq[32:]).all()


def test_slots_outside_write_nothing_and_bad_blocks_are_nan():
    x = np.full((3, 1, 32), 0x3F80, np.uint16)
    x[2, 0, 5] = 0x7F80
    c0, s0 = np.full((1, 1, 16, 32), 7, np.uint8), np.full((1, 1, 16, 1), 9, np.uint8)
    c, s = A.write(x, [-1, 16, 3], c0, s0)
    assert s[0, 0, 3, 0] == 0xFF and np.all(c[0, 0, 3] == 0x7F)
    c[0, 0, 3], s[0, 0, 3] = 7, 9
    assert np.array_equal(c, c0) and np.array_equal(s, s0)
