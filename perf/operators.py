"""The mixture-of-experts operators and the block-128 linear: cases, plain forms and the framework's calls.

Four operators, by a case's "op":

* ``route``: router logits [T, E] -> the k experts of each token, their weights, and the token slots grouped by expert.
* ``grouped``: every row times its own expert's FP8 weight, the rows ragged over the experts; the weight in MXFP8
  (E8M0 scale per 32 along K) or with FP32 scales per 128 x 128 block.  With ``act`` the input is [gate | up] and the
  product takes silu(gate) * up.
* ``combine``: the experts' rows joined per token with the router's weights, plus a shared expert's row.
* ``block128``: the dense FP8 linear with FP32 scales per 128 x 128 block of the weight.

Activations arrive in BF16 and are quantised inside the operator, per row and scale block, before the product; that
rounding is part of the operators' definition, so the plain form and the 64-bit form make it too.
"""

import math

import numpy as np
import torch

own = False

SOFTMAX, SIGMOID = "softmax", "sigmoid"
FP8_MAX = 448.0           # largest finite e4m3 value
AMAX_FLOOR = 2.0 ** -96   # smallest block maximum an FP32 activation scale is made from


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of a handful of sequences: the router's latency
        {"name": "route decode", "op": "route", "T": 4, "E": 64, "k": 6, "score": SOFTMAX, "bias": False, "dtype": "bf16"},
        # a prefill chunk through a wide router with a balancing bias
        {"name": "route prefill", "op": "route", "T": 8192, "E": 256, "k": 8, "score": SIGMOID, "bias": True, "dtype": "f32"},
        # a single token's expert rows joined
        {"name": "combine token", "op": "combine", "T": 1, "k": 8, "N": 5120, "shared": True},
        # a prefill chunk's expert rows joined
        {"name": "combine prefill", "op": "combine", "T": 8192, "k": 8, "N": 5120, "shared": True},
        # gate and up projections of one decoded token: 8 experts' weights are streamed
        {"name": "gate-up token", "op": "grouped", "T": 1, "E": 32, "k": 8, "N": 4608, "K": 5120, "act": False, "scales": "mx"},
        # down projection of a decode batch: a few dozen ragged rows for each expert
        {"name": "down batch", "op": "grouped", "T": 193, "E": 32, "k": 8, "N": 5120, "K": 2304, "act": True, "scales": "mx"},
        # down projection of a tensor-parallel quarter, whose K is no multiple of 128
        {"name": "down quarter", "op": "grouped", "T": 1000, "E": 64, "k": 6, "N": 5120, "K": 576, "act": True, "scales": "mx"},
        # gate and up projections of a prefill chunk
        {"name": "gate-up prefill", "op": "grouped", "T": 8192, "E": 32, "k": 8, "N": 4608, "K": 5120, "act": False, "scales": "mx"},
        # experts of a checkpoint with FP32 block scales, a prefill chunk
        {"name": "gate-up fp32 scales", "op": "grouped", "T": 4096, "E": 16, "k": 4, "N": 2304, "K": 4096, "act": False, "scales": "f32"},
        # a dense layer of such a checkpoint: one token, a ragged medium batch with edges inside the blocks, a prefill chunk
        {"name": "dense token", "op": "block128", "M": 1, "N": 5120, "K": 2304},
        {"name": "dense odd", "op": "block128", "M": 777, "N": 1040, "K": 4112},
        {"name": "dense prefill", "op": "block128", "M": 8192, "N": 5120, "K": 4096},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "combine", "grouped", "grouped", "block128"])
    if op == "route":
        e = rng.randint(8, 512)
        return {"op": op, "T": _log(rng, 1, 8192), "E": e, "k": rng.randint(1, min(12, e)), "score": rng.choice([SOFTMAX, SIGMOID]),
                "bias": rng.random() < 0.5, "dtype": rng.choice(["bf16", "f32"])}
    if op == "combine":
        return {"op": op, "T": _log(rng, 1, 8192), "k": rng.randint(1, 8), "N": 8 * _log(rng, 32, 640), "shared": rng.random() < 0.5}
    if op == "grouped":
        e = rng.randint(2, 64)
        scales = rng.choice(["mx", "f32"])
        step = 32 if scales == "mx" else 16
        return {"op": op, "T": _log(rng, 1, 4096), "E": e, "k": rng.randint(1, min(8, e)), "N": 16 * _log(rng, 8, 320),
                "K": step * _log(rng, 4, 4608 // step), "act": rng.random() < 0.5, "scales": scales}
    return {"op": op, "M": _log(rng, 1, 8192), "N": 16 * _log(rng, 4, 320), "K": 16 * _log(rng, 8, 256)}


def _ceil(a, b):
    return -(-a // b)


def _active(case):
    """Experts that at least one of T tokens picks, on average, when each picks k of E evenly."""
    return case["E"] * (1.0 - (1.0 - case["k"] / case["E"]) ** case["T"])


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": T * E * size + (4 * E if case["bias"] else 0) + T * k * 16 + 4 * (E + 1), "flops": 4 * T * E}
    if op == "combine":
        T, k, N = case["T"], case["k"], case["N"]
        return {"bytes": T * N * 2 * (k + 1 + int(case["shared"])) + T * k * 8, "flops": 2 * T * k * N}
    if op == "grouped":
        S, N, K = case["T"] * case["k"], case["N"], case["K"]
        rows = S if case["act"] else case["T"]
        scale = N * K / 32 if case["scales"] == "mx" else 4 * _ceil(N, 128) * _ceil(K, 128)
        return {"bytes": rows * K * (4 if case["act"] else 2) + _active(case) * (N * K + scale) + S * N * 2, "flops": 2 * S * N * K}
    M, N, K = case["M"], case["N"], case["K"]
    return {"bytes": M * K * 2 + N * K + 4 * _ceil(N, 128) * _ceil(K, 128) + M * N * 2, "flops": 2 * M * N * K}


# ----------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(g, rows, width):
    """Standard normal, one channel in a hundred 20 times as large, in BF16."""
    x = torch.randn((rows, width), generator=g, device="cuda", dtype=torch.float32)
    big = torch.rand((width,), generator=g, device="cuda") < 0.01
    return (x * torch.where(big, 20.0, 1.0)).to(torch.bfloat16)


def _codes(g, shape):
    """e4m3 codes over all finite values (0x7F and 0xFF are NaN)."""
    c = torch.randint(0, 254, shape, generator=g, device="cuda", dtype=torch.uint8)
    return c + (c >= 0x7F).to(torch.uint8)


def _routing(g, T, E, k):
    """Ids of k different experts for each token, some experts more popular than others."""
    liking = 0.5 * torch.randn((E,), generator=g, device="cuda")
    return torch.topk(torch.randn((T, E), generator=g, device="cuda") + liking, k, dim=1).indices


def _group(ids, E):
    """The flat slots sorted by expert (stable), and where each expert's rows begin."""
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    offsets = torch.searchsorted(flat[order], torch.arange(E + 1, device=flat.device))
    return offsets.to(torch.int32), order.to(torch.int32)


def _weights(g, case, lead):
    N, K = case["N"], case["K"]
    w = _codes(g, lead + (N, K))
    if case.get("scales", "f32") == "mx":
        ws = torch.randint(117, 124, lead + (N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    else:
        ws = 1e-3 * (0.5 + 1.5 * torch.rand(lead + (_ceil(N, 128), _ceil(K, 128)), generator=g, device="cuda"))
    return w, ws


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"op": op, "case": dict(case)}
    if op == "route":
        T, E = case["T"], case["E"]
        logits = 1.5 * torch.randn((T, E), generator=g, device="cuda")
        s["logits"] = logits.to(torch.bfloat16) if case["dtype"] == "bf16" else logits
        s["bias"] = 0.1 * torch.randn((E,), generator=g, device="cuda") if case["bias"] else None
    elif op == "combine":
        T, k, N = case["T"], case["k"], case["N"]
        s["y"] = torch.randn((T * k, N), generator=g, device="cuda").to(torch.bfloat16)
        s["slot_row"] = torch.randperm(T * k, generator=g, device="cuda").to(torch.int32).view(T, k)
        s["weights"] = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), dim=1)
        s["shared"] = torch.randn((T, N), generator=g, device="cuda").to(torch.bfloat16) if case["shared"] else None
    elif op == "grouped":
        T, E, k, K = case["T"], case["E"], case["k"], case["K"]
        s["offsets"], s["row_slot"] = _group(_routing(g, T, E, k), E)
        # the largest group, which a plain form pads the others to
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())
        # after the activation, rows are the expert's own; before it they are the tokens'
        s["x"] = _activations(g, T * k, 2 * K) if case["act"] else _activations(g, T, K)
        s["w"], s["w_scale"] = _weights(g, case, (E,))
    else:
        s["x"] = _activations(g, case["M"], case["K"])
        s["w"], s["w_scale"] = _weights(g, case, ())
    return s


# ------------------------------------------------------------- plain forms

def _pow2(e):
    """2^e in FP32 for int32 e in [-126, 127]."""
    return ((e + 127) << 23).view(torch.float32)


def _e4m3(v):
    """FP32 values rounded to e4m3, saturating, as FP32."""
    return v.clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn).to(torch.float32)


def _blocks(x, block):
    """[rows, K] -> FP32 [rows, ceil(K / block), block], padded with zeros."""
    rows, K = x.shape
    x = torch.nn.functional.pad(x.to(torch.float32), (0, _ceil(K, block) * block - K))
    return x.view(rows, -1, block)


def _quantise_mx(x):
    """The values an MXFP8 activation stands for: per row and 32 consecutive K, e = ceil(log2(amax / 448)), codes of x / 2^e."""
    K = x.shape[1]
    b = _blocks(x, 32)
    m, e = torch.frexp(b.abs().amax(dim=2, keepdim=True))         # amax = m 2^e, m in [0.5, 1); 448 = 1.75 * 2^8
    e = (e.to(torch.int32) - 9 + (m > 0.875).to(torch.int32)).clamp(-126, 119)
    return (_e4m3(b * _pow2(-e)) * _pow2(e)).view(x.shape[0], -1)[:, :K]


def _quantise_f32(x):
    """The values of an activation with one FP32 scale amax / 448 per row and 128 consecutive K."""
    K = x.shape[1]
    b = _blocks(x, 128)
    amax = b.abs().amax(dim=2, keepdim=True).clamp_min(AMAX_FLOOR)
    return (_e4m3(b * (FP8_MAX / amax)) * (amax / FP8_MAX)).view(x.shape[0], -1)[:, :K]


def _dequantise(w, w_scale):
    """FP32 values of e4m3 codes [.., N, K] with E8M0 scales per 32 K (uint8) or FP32 scales per 128 x 128 block."""
    N, K = w.shape[-2:]
    v = w.view(torch.float8_e4m3fn).to(torch.float32)
    if w_scale.dtype == torch.uint8:
        return v * _pow2(w_scale.to(torch.int32) - 127).repeat_interleave(32, dim=-1)
    return v * w_scale.repeat_interleave(128, dim=-2)[..., :N, :].repeat_interleave(128, dim=-1)[..., :K]


def _swiglu(x):
    """silu(gate) * up of rows [gate | up], rounded to BF16 as the activation's storage type."""
    K = x.shape[1] // 2
    gate, up = x[:, :K].to(torch.float32), x[:, K:].to(torch.float32)
    return (gate / (1.0 + torch.exp(-gate)) * up).to(torch.bfloat16)


def _route(logits, bias, k, score):
    T, E = logits.shape
    # FP32 scores when the logits themselves decide; 64 bits where scores are compared, so that no rounding decides
    l = logits.to(torch.float32 if bias is None else torch.float64)
    if score == SOFTMAX:
        p = torch.exp(l - l.amax(dim=1, keepdim=True))
        p = p / p.sum(dim=1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    key = l if bias is None else p + bias.to(torch.float64)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    weights = torch.gather(p, 1, ids)
    weights = (weights / weights.sum(dim=1, keepdim=True) * 2.5).to(torch.float32)
    offsets, row_slot = _group(ids, E)
    slot_row = torch.empty_like(row_slot)
    slot_row[row_slot.to(torch.int64)] = torch.arange(T * k, device=ids.device, dtype=torch.int32)
    return ids.to(torch.int32), weights, offsets, row_slot, slot_row.view(T, k)


def _grouped(s):
    c = s["case"]
    E, k, N, most = c["E"], c["k"], c["N"], s["most"]
    S = s["row_slot"].numel()
    row = torch.arange(S, device="cuda")
    offsets = s["offsets"].to(torch.int64)
    expert = torch.searchsorted(offsets[1:].contiguous(), row, right=True)
    x = _swiglu(s["x"]) if c["act"] else s["x"]
    q = _quantise_mx(x) if c["scales"] == "mx" else _quantise_f32(x)
    if not c["act"]:
        q = q[s["row_slot"].to(torch.int64) // k]
    if S < E:                                   # fewer rows than experts: each row with its expert's weight
        w = _dequantise(s["w"][expert], s["w_scale"][expert])
        return torch.matmul(w, q.unsqueeze(2)).squeeze(2).to(torch.bfloat16)
    place = expert * most + row - offsets[expert]
    padded = torch.zeros((E * most, q.shape[1]), dtype=torch.float32, device="cuda")
    padded[place] = q
    w = _dequantise(s["w"], s["w_scale"])
    out = torch.matmul(padded.view(E, most, -1), w.transpose(1, 2))
    return out.view(E * most, N)[place].to(torch.bfloat16)


def _combine(y, slot_row, weights, shared):
    out = (y[slot_row.to(torch.int64)].to(torch.float32) * weights.unsqueeze(2)).sum(dim=1)
    if shared is not None:
        out = out + shared.to(torch.float32)
    return out.to(torch.bfloat16)


def run(state):
    s, c, op = state, state["case"], state["op"]
    if own:
        import mx_scaled_fp8_amd as mx
        if op == "route":
            score = mx.MX_ROUTE_SOFTMAX if c["score"] == SOFTMAX else mx.MX_ROUTE_SIGMOID
            return mx.mx_moe_route(s["logits"], c["k"], bias=s["bias"], score=score, renormalize=True, scale=2.5)
        if op == "combine":
            return mx.mx_moe_combine(s["y"], s["slot_row"], s["weights"], shared=s["shared"])
        if op == "grouped":
            if c["act"]:
                return mx.mx_grouped_linear(s["x"], s["w"], s["w_scale"], s["offsets"], act=mx.MX_ACT_SWIGLU)
            return mx.mx_grouped_linear(s["x"], s["w"], s["w_scale"], s["offsets"], row_slot=s["row_slot"], k=c["k"])
        return mx.mx_linear_block128(s["x"], s["w"], s["w_scale"])
    if op == "route":
        return _route(s["logits"], s["bias"], c["k"], c["score"])
    if op == "combine":
        return _combine(s["y"], s["slot_row"], s["weights"], s["shared"])
    if op == "grouped":
        return _grouped(s)
    return torch.matmul(_quantise_f32(s["x"]), _dequantise(s["w"], s["w_scale"]).t()).to(torch.bfloat16)


# ------------------------------------------------------------- in 64 bits
#
# Written from the definitions: e4m3 by its grid (spacing 2^(floor(log2|v|) - 3), at least 2^-9), E8M0 by powers of
# two, the products expert by expert.

def _table():
    """The 256 e4m3 values from their bit fields."""
    c = np.arange(256)
    field, frac = (c >> 3) & 15, c & 7
    v = np.where(field == 0, frac * 2.0 ** -9, (8 + frac) * 2.0 ** (field.astype(np.float64) - 10))
    v = np.where((c & 127) == 127, np.nan, v)
    return torch.from_numpy(np.where(c >= 128, -v, v)).cuda()


def _grid64(v):
    v = v.clamp(-448.0, 448.0)
    _, e = torch.frexp(v.abs().clamp_min(2.0 ** -6))
    step = torch.exp2((e - 4).to(torch.float64))
    return torch.round(v / step) * step


def _quantised64(x, scales):
    out = torch.empty_like(x)
    block = 32 if scales == "mx" else 128
    for k0 in range(0, x.shape[1], block):
        b = x[:, k0:k0 + block]
        amax = b.abs().amax(dim=1, keepdim=True)
        if scales == "mx":
            unit = torch.exp2(torch.ceil(torch.log2(amax.clamp_min(2.0 ** -118) / 448.0)))
        else:
            unit = amax.clamp_min(AMAX_FLOOR) / 448.0
        out[:, k0:k0 + block] = _grid64(b / unit) * unit
    return out


def _weight64(w, w_scale, table):
    v = table[w.to(torch.int64)]
    n = torch.arange(w.shape[0], device="cuda")
    k = torch.arange(w.shape[1], device="cuda")
    if w_scale.dtype == torch.uint8:
        return v * torch.exp2(w_scale.to(torch.float64) - 127.0)[:, k // 32]
    return v * w_scale.to(torch.float64)[n // 128][:, k // 128]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "route":
        l = s["logits"].to(torch.float64)
        p = torch.softmax(l, dim=1) if case["score"] == SOFTMAX else torch.sigmoid(l)
        ids = torch.sort(l if s["bias"] is None else p + s["bias"].to(torch.float64), dim=1, descending=True, stable=True).indices[:, :case["k"]]
        chosen = p.gather(1, ids)
        return None, 2.5 * chosen / chosen.sum(dim=1, keepdim=True), None, None, None
    if op == "combine":
        out = s["shared"].to(torch.float64) if case["shared"] else torch.zeros((case["T"], case["N"]), dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            out = out + s["weights"][:, j:j + 1].to(torch.float64) * s["y"][s["slot_row"][:, j].to(torch.int64)].to(torch.float64)
        return out
    table = _table()
    if op == "block128":
        return _quantised64(s["x"].to(torch.float64), "f32") @ _weight64(s["w"], s["w_scale"], table).t()
    x = s["x"].to(torch.float64)
    if case["act"]:
        gate, up = x[:, :case["K"]], x[:, case["K"]:]
        x = (gate * torch.sigmoid(gate) * up).to(torch.bfloat16).to(torch.float64)
    q = _quantised64(x, case["scales"])
    if not case["act"]:
        q = q[s["row_slot"].to(torch.int64) // case["k"]]
    out = torch.empty((q.shape[0], case["N"]), dtype=torch.float64, device="cuda")
    begins = s["offsets"].tolist()
    for e in range(case["E"]):
        if begins[e + 1] > begins[e]:
            out[begins[e]:begins[e + 1]] = q[begins[e]:begins[e + 1]] @ _weight64(s["w"][e], s["w_scale"][e], table).t()
    return out
