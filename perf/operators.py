"""Cases of the microscaled 4-bit (MXFP4) operators and of the token dispatch around the experts.

Five operators, each reached through weight_only_bit_amd's public calls:

  quantize   rows of f32 or bf16 values to MXFP4 (e2m1 codes, one power-of-two scale per 32) and
             back to the bf16 values that the codes stand for
  product    y = x W^T with MXFP4 weights; activations bf16, or quantised to MXFP4 in the call
  experts    the grouped product over tokens sorted by expert, both operands MXFP4: gate+up with
             SiLU(gate) * up (tokens gathered by the product) or down (rows in expert order)
  sort       token rows into expert order (routing sort, positions, rows); in training also the
             gradient: every token's sum over its rows' gradients
  back       sorted rows back to their tokens, weighted; in training also the gradients of the
             rows and of the weights
"""
import math

import torch

own = False

# Magnitudes of the eight e2m1 codes (the ninth bit pattern on is the same with the sign).
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # a layer's weights, as a checkpoint holds them, packed once
        {"name": "quantize weights f32", "op": "quantize", "dtype": "f32", "n": 8192, "k": 8192},
        # a few tokens' activations before a decode product: latency
        {"name": "quantize rows bf16", "op": "quantize", "dtype": "bf16", "n": 17, "k": 4096},
        # one token through one linear layer
        {"name": "product 1 token", "op": "product", "act": "mx", "m": 1, "n": 4096, "k": 4096},
        # a decode batch against MXFP4 weights, activations left in bf16
        {"name": "product 8 rows bf16", "op": "product", "act": "bf16", "m": 8, "n": 4096, "k": 4096},
        # a ragged chunk of a prompt: odd rows, odd outputs, k that is no multiple of 128
        {"name": "product ragged", "op": "product", "act": "mx", "m": 333, "n": 1111, "k": 4160},
        # a prompt of 4096 tokens through a square layer
        {"name": "product prompt", "op": "product", "act": "mx", "m": 4096, "n": 8192, "k": 8192},
        # the decode step of the 64-expert layer: 32 tokens, top-8
        {"name": "experts decode", "op": "experts", "kind": "gate_up", "t": 32, "topk": 8, "experts": 64,
         "n": 3584, "k": 8192, "skew": 0.0},
        # its prompt step, experts loaded unevenly
        {"name": "experts prompt", "op": "experts", "kind": "down", "t": 4096, "topk": 8, "experts": 64,
         "n": 8192, "k": 3584, "skew": 1.1},
        # the dispatch of a decode batch
        {"name": "sort decode", "op": "sort", "t": 32, "topk": 8, "experts": 64, "hidden": 8192,
         "dtype": "bf16", "grad": False, "skew": 0.0},
        # a training batch: tokens to expert order and the gradient back
        {"name": "sort training", "op": "sort", "t": 4096, "topk": 8, "experts": 64, "hidden": 8192,
         "dtype": "bf16", "grad": True, "skew": 1.1},
        # the weighted sum of a decode batch
        {"name": "back decode", "op": "back", "t": 32, "topk": 8, "hidden": 8192, "experts": 64,
         "dtype": "bf16", "grad": False, "skew": 0.0},
        # a training batch: the weighted sum and both gradients
        {"name": "back training", "op": "back", "t": 4096, "topk": 8, "hidden": 8192, "experts": 64,
         "dtype": "bf16", "grad": True, "skew": 1.1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "product", "product", "experts", "experts", "sort", "back"))
    if op == "quantize":
        return {"op": op, "dtype": rng.choice(("f32", "bf16")), "n": _log(rng, 1, 8192),
                "k": 64 * _log(rng, 1, 128)}
    if op == "product":
        return {"op": op, "act": rng.choice(("mx", "mx", "bf16")), "m": _log(rng, 1, 4096),
                "n": _log(rng, 16, 8192), "k": 64 * _log(rng, 4, 128)}
    experts = rng.choice((4, 8, 16, 64))
    topk = rng.randint(1, min(8, experts))
    skew = rng.choice((0.0, 1.1))
    if op == "experts":
        kind = rng.choice(("gate_up", "down"))
        return {"op": op, "kind": kind, "t": _log(rng, 1, 2048), "topk": topk, "experts": experts,
                "n": _log(rng, 64, 3584), "k": 64 * _log(rng, 4, 112), "skew": skew}
    return {"op": op, "t": _log(rng, 1, 4096), "topk": topk, "experts": experts, "hidden": _log(rng, 64, 8192),
            "dtype": rng.choice(("bf16", "bf16", "f32")), "grad": rng.random() < 0.5, "skew": skew}


def work(case):
    op = case["op"]
    if op == "quantize":
        v = case["n"] * case["k"]
        e = 4 if case["dtype"] == "f32" else 2
        return {"bytes": v * (e + 17 / 32 + 2), "flops": 3 * v}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 2 * m * k + n * k * 17 / 32 + 2 * m * n, "flops": 2 * m * n * k}
    t, topk, experts = case["t"], case["topk"], case["experts"]
    p = t * topk
    if op == "experts":
        n, k = case["n"], case["k"]
        touched = experts * (1 - (1 - topk / experts) ** t)
        two = 2 if case["kind"] == "gate_up" else 1
        rows = t if case["kind"] == "gate_up" else p
        return {"bytes": 2 * rows * k + two * touched * n * k * 17 / 32 + 2 * p * n, "flops": two * 2 * p * n * k}
    e = 4 if case["dtype"] == "f32" else 2
    h = case["hidden"]
    if op == "sort":
        b = (t + p) * h * e + 12 * p
        return {"bytes": b * (2 if case["grad"] else 1), "flops": p * h if case["grad"] else p}
    b = (t + p) * h * e + 8 * p
    return {"bytes": b + ((t + 2 * p) * h * e if case["grad"] else 0), "flops": 2 * p * h * (3 if case["grad"] else 1)}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _activations(g, rows, k):
    # unit normal values with a few channels ten times larger, as hidden states have them
    x = _normal(g, rows, k)
    x[:, torch.randperm(k, generator=g, device="cuda")[: max(1, k // 512)]] *= 10.0
    return x.to(torch.bfloat16)


def _routing(g, case):
    t, topk, experts = case["t"], case["topk"], case["experts"]
    bias = -case["skew"] * torch.log(torch.arange(1, experts + 1, device="cuda", dtype=torch.float32))
    top = torch.topk(_normal(g, t, experts) + bias, topk, dim=1)
    return top.indices.to(torch.int32).contiguous(), torch.softmax(top.values, 1).contiguous()


def _packed(g, experts, n, k):
    """Normal weights in MXFP4: (codes [E, n, k/2], scale bytes [E, n, k/32])."""
    codes = torch.empty((experts, n, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((experts, n, k // 32), dtype=torch.uint8, device="cuda")
    for e in range(experts):
        c, s = _encode(_normal(g, n, k) * 0.02)
        codes[e] = c[:, 0::2] | (c[:, 1::2] << 4)
        scales[e] = s
    return codes, scales


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "quantize":
        if case["dtype"] == "f32":
            s["x"] = _normal(g, case["n"], case["k"]) * 0.02
        else:
            s["x"] = _activations(g, case["n"], case["k"])
    elif op == "product":
        s["x"] = _activations(g, case["m"], case["k"])
        s["w"] = _weight(_packed(g, 1, case["n"], case["k"]))
    else:
        ids, wts = _routing(g, case)
        p = ids.numel()
        # the routing plan: pairs sorted by expert (stable), every expert's first row, and the
        # row of every pair
        pairs = torch.sort(ids.reshape(-1), stable=True).indices.to(torch.int32)
        positions = torch.empty_like(pairs)
        positions[pairs.long()] = torch.arange(p, dtype=torch.int32, device="cuda")
        offsets = torch.zeros(case["experts"] + 1, dtype=torch.int32, device="cuda")
        offsets[1:] = torch.cumsum(torch.bincount(ids.reshape(-1), minlength=case["experts"]), 0)
        if op == "experts":
            s["x"] = _activations(g, case["t"] if case["kind"] == "gate_up" else p, case["k"])
            s["offsets"], s["pairs"] = offsets, pairs
            s["w"] = _weight(_packed(g, case["experts"], case["n"], case["k"]))
            if case["kind"] == "gate_up":
                s["up"] = _weight(_packed(g, case["experts"], case["n"], case["k"]))
        else:
            dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
            h = case["hidden"]
            if op == "sort":
                s["ids"] = ids
                s["x"] = _activations(g, case["t"], h).to(dt)
                if case["grad"]:
                    s["d_rows"] = (_normal(g, p, h) * 1e-2).to(dt)
            else:
                s["positions"], s["weights"] = positions.view(case["t"], case["topk"]), wts
                s["rows"] = _normal(g, p, h).to(dt)
                if case["grad"]:
                    s["dy"] = (_normal(g, case["t"], h) * 1e-2).to(dt)
    return s


def _weight(arrays):
    """A packed weight, as a user's program holds it: the arrays, and the handle around them."""
    return {"codes": arrays[0], "scales": arrays[1], "handle": None}


def _handle(w):
    if w["handle"] is None:
        import weight_only_bit_amd as wq

        e, n, half = w["codes"].shape
        w["handle"] = wq.PackedWeight(wq.FMT_MXFP4, n, 2 * half, e, 32, codes=w["codes"], qscale=w["scales"])
    return w["handle"]


# ---------------------------------------------------------------------------------------------
# plain form
# ---------------------------------------------------------------------------------------------

def _encode(x):
    """(code of every value, scale byte of every block of 32), OCP microscaling e2m1 rules."""
    n, k = x.shape
    v = x.float().view(n, k // 32, 32)
    exponent = torch.frexp(v.abs().amax(2)).exponent - 1  # floor(log2 |max|)
    byte = (exponent - 2 + 127).clamp(0, 254)
    u = torch.ldexp(v, (127 - byte).unsqueeze(2)).view(n, k)
    a = u.abs()
    # half way between two codes, the one with the even code is taken
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return code.to(torch.uint8) | (torch.signbit(u).to(torch.uint8) << 3), byte.to(torch.uint8)


def _values(code, byte):
    """fp32 values of codes [..., k] with scale bytes [..., k/32]."""
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=code.device)
    v = table[code.int()].view(*byte.shape, 32)
    return torch.ldexp(v, (byte.int() - 127).unsqueeze(-1)).view(code.shape)


def _unpacked(w):
    c = w["codes"]
    return _values(torch.stack((c & 15, c >> 4), -1).view(*c.shape[:-1], 2 * c.shape[-1]), w["scales"])


def _fake_quantized(x):
    return _values(*_encode(x))


def _grouped(x, w, offsets, room):
    """Rows x [p, k] in expert order times their expert's matrix w [E, n, k]: [p, n], in fp32.
    room: the rows that one expert gets at most (one per token)."""
    p, experts = x.shape[0], w.shape[0]
    row = torch.arange(p, device=x.device)
    e = torch.searchsorted(offsets[1:].long(), row, right=True)
    slot = row - offsets.long()[e]
    padded = torch.zeros((experts, x.shape[1], room), device=x.device)
    padded[e, :, slot] = x
    return torch.bmm(w, padded)[e, :, slot]


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import weight_only_bit_amd as wq

        if op == "quantize":
            return wq.wq_dequantize(wq.wq_quantize_mx(state["x"])).view(torch.bfloat16)
        if op == "product":
            w = _handle(state["w"])
            if case["act"] == "bf16":
                return wq.wq_gemm(state["x"], w)
            return wq.wq_gemm_mx(wq.wq_quantize_mx(state["x"]), w)
        if op == "experts":
            x = wq.wq_quantize_mx(state["x"])
            if case["kind"] == "gate_up":
                return wq.wq_moe_gate_up_mx(x, state["offsets"], state["pairs"], case["topk"], _handle(state["w"]),
                                            _handle(state["up"]))
            return wq.wq_moe_down_mx(x, state["offsets"], _handle(state["w"]))
        if op == "sort":
            offsets, pairs = wq.wq_moe_route(state["ids"], case["experts"])
            positions = wq.wq_moe_positions(state["ids"], offsets, pairs)
            out = {"rows": wq.wq_moe_permute(state["x"], positions), "offsets": offsets, "positions": positions}
            if case["grad"]:
                out["dx"] = wq.wq_moe_unpermute(state["d_rows"], positions)
            return out
        out = {"y": wq.wq_moe_unpermute(state["rows"], state["positions"], state["weights"])}
        if case["grad"]:
            out["d_rows"], out["d_weights"] = wq.wq_moe_unpermute_grad(state["dy"], state["rows"], state["positions"],
                                                                       state["weights"])
        return out

    if op == "quantize":
        return _fake_quantized(state["x"]).to(torch.bfloat16)[None]
    if op == "product":
        x = state["x"].float() if case["act"] == "bf16" else _fake_quantized(state["x"])
        return (x @ _unpacked(state["w"])[0].t()).to(torch.bfloat16)
    if op == "experts":
        x = _fake_quantized(state["x"])
        if case["kind"] == "down":
            return _grouped(x, _unpacked(state["w"]), state["offsets"], case["t"]).to(torch.bfloat16)
        x = x[state["pairs"].long() // case["topk"]]
        gate = _grouped(x, _unpacked(state["w"]), state["offsets"], case["t"])
        up = _grouped(x, _unpacked(state["up"]), state["offsets"], case["t"])
        return (gate / (1 + torch.exp(-gate)) * up).to(torch.bfloat16)
    t, topk = case["t"], case["topk"]
    if op == "sort":
        ids = state["ids"].reshape(-1)
        order = torch.sort(ids, stable=True).indices
        positions = torch.empty_like(ids)
        positions[order] = torch.arange(t * topk, dtype=torch.int32, device=ids.device)
        counts = (ids[:, None] == torch.arange(case["experts"], device=ids.device)).sum(0)
        offsets = torch.cat((counts.new_zeros(1), torch.cumsum(counts, 0))).to(torch.int32)
        out = {"rows": state["x"][order // topk], "offsets": offsets, "positions": positions.view(t, topk)}
        if case["grad"]:
            out["dx"] = state["d_rows"].float()[positions.long()].view(t, topk, -1).sum(1).to(state["x"].dtype)
        return out
    at = state["positions"].long()
    rows, weights = state["rows"].float()[at], state["weights"]
    out = {"y": (rows * weights[:, :, None]).sum(1).to(state["rows"].dtype)}
    if case["grad"]:
        dy = state["dy"].float()
        d_rows = torch.empty_like(state["rows"])
        d_rows[at] = (weights[:, :, None] * dy[:, None, :]).to(d_rows.dtype)
        out["d_rows"], out["d_weights"] = d_rows, (rows * dy[:, None, :]).sum(2)
    return out


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------

def _exact_encode(x):
    """The e2m1 values times their block's scale, nearest value with ties to the even code."""
    n, k = x.shape
    v = x.double().view(n, k // 32, 32)
    top = v.abs().amax(2, keepdim=True)
    floor = torch.floor(torch.log2(top.clamp_min(2.0 ** -130)))
    floor = floor - (torch.exp2(floor) > top).double() + (torch.exp2(floor + 1) <= top).double()
    scale = torch.exp2((floor - 2).clamp(-127, 127))
    a = (v / scale).abs()
    # the grid's step is 1/2 below 2, 1 below 4 and 2 above; round() takes ties to even multiples
    step = 0.5 + 0.5 * (a >= 2) + 1.0 * (a >= 4)
    q = (torch.round(a / step) * step).clamp_max(6.0)
    return (torch.where(v < 0, -q, q) * scale).view(n, k)


def _exact_matrix(w, e):
    c = w["codes"][e].to(torch.int64)
    bits = torch.empty((c.shape[0], 2 * c.shape[1]), dtype=torch.int64, device=c.device)
    bits[:, 0::2], bits[:, 1::2] = c % 16, c // 16
    exponent, fraction = (bits // 2) % 4, bits % 2
    size = torch.where(exponent == 0, 0.5 * fraction, (1 + 0.5 * fraction) * torch.exp2((exponent - 1).double()))
    value = torch.where(bits >= 8, -size, size)
    return value * torch.exp2(w["scales"][e].double() - 127).repeat_interleave(32, 1)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_encode(state["x"])[None]
    if op == "product":
        x = state["x"].double() if case["act"] == "bf16" else _exact_encode(state["x"])
        return x @ _exact_matrix(state["w"], 0).t()
    if op == "experts":
        x = _exact_encode(state["x"])
        at = state["offsets"].tolist()
        out = []
        for e in range(case["experts"]):
            rows = torch.arange(at[e], at[e + 1], device=x.device)
            if case["kind"] == "gate_up":
                rows = state["pairs"][rows].long().div(case["topk"], rounding_mode="floor")
            a = x[rows] @ _exact_matrix(state["w"], e).t()
            if case["kind"] == "gate_up":
                a = a * torch.sigmoid(a) * (x[rows] @ _exact_matrix(state["up"], e).t())
            out.append(a)
        return torch.cat(out)
    t, topk = case["t"], case["topk"]
    if op == "sort":
        ids = state["ids"].long()
        pair = torch.arange(t * topk, device=ids.device)
        positions = torch.empty(t * topk, dtype=torch.int64, device=ids.device)
        order = torch.argsort(ids.reshape(-1) * (t * topk) + pair)
        positions[order] = pair
        counts = torch.bincount(ids.reshape(-1), minlength=case["experts"])
        out = {"rows": state["x"].double()[order.div(topk, rounding_mode="floor")],
               "offsets": torch.cumsum(torch.cat((counts[:1] * 0, counts)), 0).to(torch.int32),
               "positions": positions.view(t, topk).to(torch.int32)}
        if case["grad"]:
            owner = torch.empty_like(order)
            owner[positions] = pair.div(topk, rounding_mode="floor")
            out["dx"] = torch.zeros(t, case["hidden"], dtype=torch.float64, device=ids.device).index_add_(
                0, owner, state["d_rows"].double())
        return out
    at, w, rows = state["positions"].long(), state["weights"].double(), state["rows"].double()
    out = {"y": sum(w[:, j, None] * rows[at[:, j]] for j in range(topk))}
    if case["grad"]:
        dy = state["dy"].double()
        d_rows = torch.zeros_like(rows)
        for j in range(topk):
            d_rows[at[:, j]] = w[:, j, None] * dy
        out["d_rows"] = d_rows
        out["d_weights"] = torch.stack([(rows[at[:, j]] * dy).sum(1) for j in range(topk)], 1)
    return out
