"""Router, grouped FP8 products, join and the block-128 linear -- oracle, test infrastructure.

A mixture-of-experts layer on this library's formats: the router's choice of
k experts per token, each chosen slot's row times its own expert's FP8 weight,
and the weighted join of the experts' rows.  The weight is in MXFP8 (E8M0 scale
per 32 consecutive K, activations by :func:`oracle.quant.group_quant`) or has
one FP32 scale per 128 x 128 block, for which an activation has one FP32 scale
amax / 448 per row and 128 consecutive K.

Written from the formulas in fp64, slot by slot and expert by expert; pinned by
hand cases and brute-force loops (tests/test_oracle_moe.py).
"""

import numpy as np

from .formats import OCP, bf16_to_f64, e4m3_decode, e4m3_encode, f64_to_bf16_rne
from .gemm import scaled_operand
from .quant import group_quant

SOFTMAX, SIGMOID = 0, 1
#: The smallest block maximum an FP32 activation scale is made from.
AMAX_FLOOR = 2.0 ** -96


def route(logits, k, bias=None, score=SOFTMAX, renormalize=True, scale=1.0):
    """logits fp64 [T, E] -> (ids [T, k], weights fp64 [T, k], offsets [E+1], row_slot [T*k], slot_row [T, k])."""
    l = np.array(logits, dtype=np.float64)
    T, E = l.shape
    l[np.isnan(l)] = -np.inf
    l = np.minimum(l, float(np.finfo(np.float32).max))
    live = l > -np.inf
    p = np.zeros((T, E))
    for t in range(T):
        if score == SOFTMAX:
            if live[t].any():
                x = np.exp(l[t] - l[t].max())
                p[t] = x / x.sum()
        else:
            with np.errstate(over="ignore"):
                p[t] = np.where(live[t], 1.0 / (1.0 + np.exp(-l[t])), 0.0)
    key = l if bias is None else p + np.asarray(bias, dtype=np.float64)
    key = np.where(live & ~np.isnan(key), key, -np.inf) + 0.0
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(p, ids, axis=1)
    if renormalize:
        total = w.sum(axis=1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    offsets, row_slot, slot_row = group(ids, E)
    return ids.astype(np.int32), w * scale, offsets, row_slot, slot_row


def group(ids, E):
    """Slots t*k+j in ascending order within each expert."""
    flat = np.asarray(ids).reshape(-1)
    row_slot = np.array([s for e in range(E) for s in np.flatnonzero(flat == e)], dtype=np.int32)
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])]).astype(np.int32)
    slot_row = np.empty(flat.size, dtype=np.int32)
    slot_row[row_slot] = np.arange(flat.size, dtype=np.int32)
    return offsets, row_slot, slot_row.reshape(np.asarray(ids).shape)


def quantise_f32(x_bits):
    """BF16 bits [R, K] -> the fp64 values of the codes times their FP32 block scales, one per row and 128 K."""
    x = bf16_to_f64(x_bits)
    out = np.empty_like(x)
    for k0 in range(0, x.shape[1], 128):
        b = x[:, k0:k0 + 128]
        bad = ~np.isfinite(b).all(axis=1, keepdims=True)
        amax = np.maximum(np.where(bad, 0.0, np.abs(np.where(np.isfinite(b), b, 0.0)).max(axis=1, keepdims=True)),
                          AMAX_FLOOR)
        q = e4m3_decode(e4m3_encode(np.where(bad, 0.0, b) * 448.0 / amax, OCP), OCP)
        sa = (amax / 448.0).astype(np.float32).astype(np.float64)
        out[:, k0:k0 + 128] = np.where(bad, np.nan, q * sa)
    return out


def quantise_mx(x_bits):
    """BF16 bits [R, K] -> the fp64 values of their MXFP8 form (OCP, block 32)."""
    q, s = group_quant(x_bits, 32, OCP)
    return scaled_operand(q, s, 32, OCP)


def weight_f32(w, w_scale):
    """W u8 [N, K] with FP32 scales [ceil(N/128), ceil(K/128)] -> fp64 [N, K]."""
    N, K = w.shape
    s = np.asarray(w_scale, dtype=np.float64)
    return e4m3_decode(w, OCP) * s[np.arange(N) // 128][:, np.arange(K) // 128]


def operands(x_bits, w, w_scale):
    """The fp64 operands (x, W) of one product; the scale's type picks the format."""
    if np.asarray(w_scale).dtype == np.uint8:
        return quantise_mx(x_bits), scaled_operand(w, w_scale, 32, OCP)
    return quantise_f32(x_bits), weight_f32(w, w_scale)


def linear_block128(x_bits, w, w_scale):
    """x BF16 [M, K] @ W^T -> fp64 [M, N]."""
    x, wv = operands(x_bits, w, np.asarray(w_scale, dtype=np.float32))
    return x @ wv.T


def swiglu(x_bits):
    """BF16 [R, 2K] = gate | up -> fp64 silu(gate) * up, unrounded."""
    x = bf16_to_f64(x_bits)
    K = x.shape[1] // 2
    g, u = x[:, :K], x[:, K:]
    with np.errstate(over="ignore", invalid="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def grouped_linear(x_bits, w, w_scale, offsets, row_slot=None, k=1, act=False):
    """Row r of expert e (offsets[e] <= r < offsets[e+1]) = x[row_slot[r] // k] @ w[e]^T in fp64 [S, N]; rows that no
    expert owns are NaN, as are rows whose source lies outside x."""
    if act:
        x_bits = f64_to_bf16_rne(swiglu(x_bits))
    src = np.arange(x_bits.shape[0]) if row_slot is None else np.where(np.asarray(row_slot) < 0, -1,
                                                                      np.asarray(row_slot) // k)
    out = np.full((src.size, w.shape[1]), np.nan)
    for e in range(w.shape[0]):
        rows = [r for r in range(offsets[e], offsets[e + 1]) if 0 <= src[r] < x_bits.shape[0]]
        if rows:
            x, wv = operands(x_bits[src[rows]], w[e], w_scale[e])
            out[rows] = x @ wv.T
    return out


def combine(y_bits, slot_row, weights, shared_bits=None):
    """shared[t] + sum_j weights[t, j] * y[slot_row[t, j]] in fp64 [T, N]; a slot without a row or of weight 0 adds nothing."""
    y = bf16_to_f64(y_bits)
    T, k = slot_row.shape
    out = bf16_to_f64(shared_bits).copy() if shared_bits is not None else np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            if 0 <= slot_row[t, j] < y.shape[0] and weights[t, j] != 0:
                out[t] = out[t] + float(weights[t, j]) * y[slot_row[t, j]]
    return out
