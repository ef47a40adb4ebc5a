"""Cases of the 8-bit integer products, of the root-mean-square norm that feeds them, and of the routing's
balance loss.

Four operators, each reached through weight_only_bit_amd's public calls:

  norm      the residual's addition and the root-mean-square norm of the sum, bf16 or f32; in training also
            the gradients of the sum (which x and the residual share) and of the norm's weight
  product   y = x W^T with INT8 weights (a scale per channel) and activations in int8 with a scale per row:
            quantised in the call, or written by the norm in front of it
  experts   the grouped product over tokens sorted by expert, both operands in int8: gate+up with
            SiLU(gate) * up (tokens gathered by the product) or down (rows in expert order)
  balance   the routing's balance loss E sum_e (share of pairs)_e (mean probability)_e with the experts'
            counts, and the gradient of the router's logits
"""
import math

import torch

own = False

EPS = 1e-6
COEFFICIENT = 0.01


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # the norm in front of a layer, a decode batch: latency
        {"name": "norm decode", "op": "norm", "dtype": "bf16", "n": 32, "k": 8192, "grad": False},
        # a training batch: the norm and its gradients, the residual stream's own gradient among them
        {"name": "norm training", "op": "norm", "dtype": "bf16", "n": 4096, "k": 8192, "grad": True},
        # odd rows of odd length in f32, as a small model trains in
        {"name": "norm ragged f32", "op": "norm", "dtype": "f32", "n": 333, "k": 1111, "grad": True},
        # one token through the norm and one linear layer
        {"name": "product 1 token", "op": "product", "source": "norm", "m": 1, "n": 4096, "k": 4096},
        # a decode batch through one linear layer, activations quantised in the call
        {"name": "product decode", "op": "product", "source": "rows", "m": 32, "n": 4096, "k": 4096},
        # a ragged chunk of a prompt: odd rows, odd outputs, k that is no multiple of 128
        {"name": "product ragged", "op": "product", "source": "rows", "m": 333, "n": 1111, "k": 4160},
        # a prompt of 4096 tokens through the norm and a square layer
        {"name": "product prompt", "op": "product", "source": "norm", "m": 4096, "n": 8192, "k": 8192},
        # the decode step of the 64-expert layer: 32 tokens, top-8
        {"name": "experts decode", "op": "experts", "kind": "gate_up", "t": 32, "topk": 8, "experts": 64,
         "n": 3584, "k": 8192, "skew": 0.0},
        # its prompt step, experts loaded unevenly
        {"name": "experts prompt", "op": "experts", "kind": "down", "t": 4096, "topk": 8, "experts": 64,
         "n": 8192, "k": 3584, "skew": 1.1},
        # a small batch over few experts: latency
        {"name": "balance small", "op": "balance", "dtype": "f32", "t": 256, "topk": 2, "experts": 8,
         "padded": 0.0, "skew": 0.0},
        # a training batch of the 64-expert layer, padded at its end
        {"name": "balance training", "op": "balance", "dtype": "bf16", "t": 4096, "topk": 8, "experts": 64,
         "padded": 0.1, "skew": 1.1},
        # the largest batch, 256 experts
        {"name": "balance large", "op": "balance", "dtype": "f32", "t": 65536, "topk": 8, "experts": 256,
         "padded": 0.0, "skew": 1.1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "norm", "product", "product", "experts", "experts", "balance", "balance"))
    if op == "norm":
        return {"op": op, "dtype": rng.choice(("bf16", "bf16", "f32")), "n": _log(rng, 1, 8192),
                "k": _log(rng, 64, 8192), "grad": rng.random() < 0.5}
    if op == "product":
        return {"op": op, "source": rng.choice(("norm", "rows")), "m": _log(rng, 1, 4096),
                "n": _log(rng, 16, 8192), "k": 64 * _log(rng, 1, 128)}
    skew = rng.choice((0.0, 1.1))
    if op == "experts":
        experts = rng.choice((4, 8, 16, 64))
        return {"op": op, "kind": rng.choice(("gate_up", "down")), "t": _log(rng, 1, 2048),
                "topk": rng.randint(1, min(8, experts)), "experts": experts, "n": _log(rng, 64, 3584),
                "k": 64 * _log(rng, 4, 112), "skew": skew}
    experts = rng.choice((4, 8, 16, 60, 64, 160, 256))
    return {"op": op, "dtype": rng.choice(("bf16", "f32")), "t": _log(rng, 1, 65536),
            "topk": rng.randint(1, min(8, experts)), "experts": experts, "padded": rng.choice((0.0, 0.1)),
            "skew": skew}


def work(case):
    op = case["op"]
    if op == "norm":
        e = 4 if case["dtype"] == "f32" else 2
        v = case["n"] * case["k"]
        # x, residual, sum, y; dy, the sum's gradient, dx (the sum is at hand); the weight and its gradient
        grad = case["grad"]
        return {"bytes": v * e * (7 if grad else 4) + case["k"] * (e + (4 if grad else 0)),
                "flops": v * (16 if grad else 5)}
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        # the activations once (with the norm: x and the residual, and the sum written), weights, outputs
        return {"bytes": (6 if case["source"] == "norm" else 2) * m * k + n * k + 2 * n + 2 * m * n,
                "flops": 2 * m * n * k}
    t, topk, experts = case["t"], case["topk"], case["experts"]
    p = t * topk
    if op == "experts":
        n, k = case["n"], case["k"]
        touched = experts * (1 - (1 - topk / experts) ** t)
        two = 2 if case["kind"] == "gate_up" else 1
        rows = t if case["kind"] == "gate_up" else p
        return {"bytes": 2 * rows * k + two * touched * n * k + 2 * p * n, "flops": two * 2 * p * n * k}
    e = 4 if case["dtype"] == "f32" else 2
    return {"bytes": 2 * t * experts * e + 4 * p, "flops": 10 * t * experts}


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
    return x


def _routing(g, case):
    t, topk, experts = case["t"], case["topk"], case["experts"]
    bias = -case["skew"] * torch.log(torch.arange(1, experts + 1, device="cuda", dtype=torch.float32))
    logits = _normal(g, t, experts) + bias
    return logits, torch.topk(logits, topk, dim=1).indices.to(torch.int32).contiguous()


def _packed(g, experts, n, k):
    """A packed weight, as a user's program holds it: int8 codes [E, n, k] of normal values whose channel's
    largest is four deviations, a bf16 scale per channel, and the handle around them."""
    codes = torch.empty((experts, n, k), dtype=torch.int8, device="cuda")
    for e in range(experts):
        codes[e] = (_normal(g, n, k) * 32).round_().clamp_(-127, 127)
    scales = ((0.8 + 0.4 * torch.rand((experts, n), generator=g, device="cuda")) * (0.02 / 32)).to(torch.bfloat16)
    return {"codes": codes, "scales": scales, "handle": None}


def _handle(w):
    if w["handle"] is None:
        import weight_only_bit_amd as wq

        e, n, k = w["codes"].shape
        w["handle"] = wq.PackedWeight(wq.FMT_INT8, n, k, e, 0, codes=w["codes"], scales=w["scales"])
    return w["handle"]


def _norm_inputs(g, s, n, k, dt):
    s["x"] = _normal(g, n, k).to(dt)
    s["residual"] = _activations(g, n, k).to(dt)
    s["weight"] = (1 + 0.1 * _normal(g, k)).to(dt)


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = {"case": case}
    if op == "norm":
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        _norm_inputs(g, s, case["n"], case["k"], dt)
        if case["grad"]:
            s["dy"] = (_normal(g, case["n"], case["k"]) * 1e-2).to(dt)
            s["d_sum"] = (_normal(g, case["n"], case["k"]) * 1e-2).to(dt)
    elif op == "product":
        if case["source"] == "norm":
            _norm_inputs(g, s, case["m"], case["k"], torch.bfloat16)
        else:
            s["x"] = _activations(g, case["m"], case["k"]).to(torch.bfloat16)
        s["w"] = _packed(g, 1, case["n"], case["k"])
    elif op == "experts":
        _, ids = _routing(g, case)
        p = ids.numel()
        # the routing plan: pairs sorted by expert (stable) and every expert's first row
        s["pairs"] = torch.sort(ids.reshape(-1), stable=True).indices.to(torch.int32)
        offsets = torch.zeros(case["experts"] + 1, dtype=torch.int32, device="cuda")
        offsets[1:] = torch.cumsum(torch.bincount(ids.reshape(-1), minlength=case["experts"]), 0)
        s["offsets"] = offsets
        s["x"] = _activations(g, case["t"] if case["kind"] == "gate_up" else p, case["k"]).to(torch.bfloat16)
        s["w"] = _packed(g, case["experts"], case["n"], case["k"])
        if case["kind"] == "gate_up":
            s["up"] = _packed(g, case["experts"], case["n"], case["k"])
    else:
        logits, s["ids"] = _routing(g, case)
        s["logits"] = logits.to(torch.float32 if case["dtype"] == "f32" else torch.bfloat16)
        tail = int(case["t"] * case["padded"])  # tokens of padding at the end have no experts
        if tail:
            s["ids"][-tail:] = -1
        s["d_loss"] = 0.5 + torch.rand((), generator=g, device="cuda")
    return s


# ---------------------------------------------------------------------------------------------
# plain form
# ---------------------------------------------------------------------------------------------

def _quantized(v):
    """(codes, largest magnitude) of rows: 127 v / max, nearest, half way to the even code.  In 64 bits:
    values next to a border between two codes."""
    v = v.double()
    top = v.abs().amax(1, keepdim=True)
    return torch.round(v * 127 / torch.where(top > 0, top, 1.0)).float(), top.float()


def _norm(state):
    """(sum of the inputs' type, its fp32 values, 1 / root mean square)."""
    total = (state["x"].float() + state["residual"].float()).to(state["x"].dtype)
    f = total.float()
    return total, f, 1 / torch.sqrt((f * f).mean(1, keepdim=True) + EPS)


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


def _unpacked(w):
    return w["codes"].float() * w["scales"].float()[:, :, None]


def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import weight_only_bit_amd as wq

        if op == "norm":
            y, total = wq.wq_rms_norm(state["x"], state["weight"], state["residual"], eps=EPS)
            out = {"y": y, "sum": total}
            if case["grad"]:
                out["dx"], out["d_weight"] = wq.wq_rms_norm_grad(state["dy"], total, state["weight"],
                                                                 state["d_sum"], eps=EPS)
            return out
        if op == "product":
            if case["source"] == "rows":
                return {"y": wq.wq_gemm_i8(wq.wq_quantize_i8(state["x"]), _handle(state["w"]))}
            rows, total = wq.wq_rms_norm_i8(state["x"], state["weight"], state["residual"], eps=EPS)
            return {"y": wq.wq_gemm_i8(rows, _handle(state["w"])), "sum": total}
        if op == "experts":
            x = wq.wq_quantize_i8(state["x"])
            if case["kind"] == "gate_up":
                return wq.wq_moe_gate_up_i8(x, state["offsets"], state["pairs"], case["topk"], _handle(state["w"]),
                                            _handle(state["up"]))
            return wq.wq_moe_down_i8(x, state["offsets"], _handle(state["w"]))
        loss, counts = wq.wq_moe_balance_loss(state["logits"], state["ids"], COEFFICIENT)
        return {"loss": loss, "counts": counts,
                "d_logits": wq.wq_moe_balance_loss_grad(state["logits"], state["ids"], counts, COEFFICIENT,
                                                        state["d_loss"])}

    if op == "norm":
        total, f, inv = _norm(state)
        w = state["weight"].float()
        hat = f * inv
        out = {"y": (hat * w).to(total.dtype), "sum": total}
        if case["grad"]:
            dy = state["dy"].float()
            g = dy * w
            dx = inv * (g - hat * (g * hat).mean(1, keepdim=True)) + state["d_sum"].float()
            out["dx"], out["d_weight"] = dx.to(total.dtype), (dy * hat).sum(0)
        return out
    if op == "product":
        out = {}
        if case["source"] == "norm":
            out["sum"], f, inv = _norm(state)
            codes, top = _quantized(f.double() * state["weight"].double())
            scale = top * inv / 127
        else:
            codes, top = _quantized(state["x"])
            scale = top / 127
        w = state["w"]
        out["y"] = (codes @ w["codes"][0].float().t() * scale * w["scales"][0].float()).to(torch.bfloat16)
        return out
    if op == "experts":
        codes, top = _quantized(state["x"])
        x = codes * (top / 127)
        if case["kind"] == "down":
            return _grouped(x, _unpacked(state["w"]), state["offsets"], case["t"]).to(torch.bfloat16)
        x = x[state["pairs"].long() // case["topk"]]
        gate = _grouped(x, _unpacked(state["w"]), state["offsets"], case["t"])
        up = _grouped(x, _unpacked(state["up"]), state["offsets"], case["t"])
        return (gate / (1 + torch.exp(-gate)) * up).to(torch.bfloat16)
    experts, ids, z = case["experts"], state["ids"], state["logits"].float()
    hit = ids[:, :, None] == torch.arange(experts, device=ids.device)
    pairs = hit.sum((0, 1))
    real = hit.any(2).any(1)
    tokens = real.sum()
    p = torch.exp(z - z.amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True) * real[:, None]
    share = experts * pairs.float() / pairs.sum().clamp_min(1)
    each = COEFFICIENT / tokens.clamp_min(1)
    mean = (share * p).sum(1, keepdim=True)
    return {"loss": each * mean.sum(), "counts": torch.cat((pairs, tokens[None])).to(torch.int32),
            "d_logits": (state["d_loss"] * each * p * (share - mean)).to(state["logits"].dtype)}


# ---------------------------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------------------------

def _exact_rows(v):
    """The values that the int8 rows of v stand for."""
    top = torch.linalg.vector_norm(v, math.inf, dim=1, keepdim=True)
    return torch.where(top > 0, torch.round(127 * v / top), 0.0) * top / 127


def _exact_norm(state):
    plain = state["x"].double() + state["residual"].double()
    stored = plain.to(state["x"].dtype).double()  # the stream is kept in the inputs' type
    return plain, stored, stored.square().mean(1, keepdim=True).add(EPS).rsqrt()


def _exact_matrix(w, e):
    return w["codes"][e].double() * w["scales"][e].double().unsqueeze(1)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        plain, r, inv = _exact_norm(state)
        w = state["weight"].double()
        out = {"y": r * inv * w, "sum": plain}
        if case["grad"]:
            dy, k = state["dy"].double(), case["k"]
            # d/dr_j of sum_i dy_i w_i r_i inv(r), inv' = -inv^3 r_j / k
            along = (dy * w * r).sum(1, keepdim=True)
            out["dx"] = dy * w * inv - along * inv ** 3 * r / k + state["d_sum"].double()
            out["d_weight"] = (dy * (r * inv)).sum(0)
        return out
    if op == "product":
        out = {}
        if case["source"] == "norm":
            out["sum"], r, inv = _exact_norm(state)
            x = _exact_rows(r * state["weight"].double()) * inv
        else:
            x = _exact_rows(state["x"].double())
        out["y"] = x @ _exact_matrix(state["w"], 0).t()
        return out
    if op == "experts":
        x = _exact_rows(state["x"].double())
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
    experts = case["experts"]
    ids = state["ids"].long()
    inside = (ids >= 0) & (ids < experts)
    counts = torch.bincount(ids[inside], minlength=experts)
    real = inside.any(1)
    tokens = int(real.sum())
    d_logits = torch.zeros_like(state["logits"], dtype=torch.float64)
    loss = torch.zeros((), dtype=torch.float64, device=ids.device)
    if tokens:
        z = state["logits"][real].double()
        share = counts.double() * experts / counts.sum()
        p = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
        loss = COEFFICIENT * torch.dot(share, p.mean(0))
        slope = state["d_loss"].double() * COEFFICIENT / tokens
        d_logits[real] = slope * (p * share - p * (p @ share)[:, None])
    return {"loss": loss, "counts": torch.cat((counts, real.sum()[None])).to(torch.int32), "d_logits": d_logits}
