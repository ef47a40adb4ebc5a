"""The int8 operators together, as a layer uses them: the norm with the residual writes int8 rows, the router's
loss and counts beside the experts' products, rows back to their tokens; eager, captured and on two streams, and
a training step through torch.autograd.Function."""
import numpy as np
import pytest

import i8_testutil as i8
import mx_testutil as mx

pytestmark = pytest.mark.gpu

E, HIDDEN, INTER, TOPK = 8, 320, 192, 2


@pytest.fixture(scope="module")
def wq():
    import torch

    import weight_only_bit_amd as wq

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    wq.lib()
    return wq


class Layer:
    """A pre-norm MoE layer in int8: weights of its own, everything on the current stream."""

    def __init__(self, wq, seed=0):
        import torch

        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")
        self.wq = wq
        self.norm = (1 + 0.2 * r(HIDDEN)).to(torch.bfloat16)
        self.router = wq.wq_quantize_i8_weight(r(E, HIDDEN))
        self.gate, self.up = (wq.wq_quantize_i8_weight(r(E, INTER, HIDDEN) * 0.1) for _ in range(2))
        self.down = wq.wq_quantize_i8_weight(r(E, HIDDEN, INTER) * 0.1)

    def __call__(self, x, residual, real=None):
        import torch

        wq = self.wq
        rows, stream = wq.wq_rms_norm_i8(x, self.norm, residual)
        logits = wq.wq_gemm_i8(rows, self.router, dtype=torch.float32)
        top = torch.topk(logits, TOPK, dim=1)
        ids = top.indices.to(torch.int32)
        if real is not None:  # padding has no experts
            ids = torch.where(real[:, None], ids, torch.full_like(ids, -1))
        weights = torch.softmax(top.values, 1)
        loss, counts = wq.wq_moe_balance_loss(logits, ids, 0.01)
        offsets, pairs = wq.wq_moe_route(ids, E)
        positions = wq.wq_moe_positions(ids, offsets, pairs)
        h = torch.zeros((ids.numel(), INTER), dtype=torch.bfloat16, device="cuda")
        wq.wq_moe_gate_up_i8(rows, offsets, pairs, TOPK, self.gate, self.up, h=h)
        hq = wq.wq_quantize_i8(h)
        d = wq.wq_moe_down_i8(hq, offsets, self.down, dtype=torch.float32)
        y = wq.wq_moe_unpermute(d, positions, weights)
        return {"rows": rows, "stream": stream, "logits": logits, "ids": ids, "weights": weights, "loss": loss,
                "counts": counts, "offsets": offsets, "pairs": pairs, "positions": positions, "h": h, "hq": hq, "d": d, "y": y,
                "d_logits": wq.wq_moe_balance_loss_grad(logits, ids, counts, 0.01)}


def _inputs(t, seed):
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn((t, HIDDEN), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]


def _weight(w):
    return w.codes.cpu().numpy(), i8.to_host(w.scales)


@pytest.mark.parametrize("t", [1, 7, 64, 700])
@pytest.mark.parametrize("padded", [False, True])
def test_layer_stage_by_stage(wq, t, padded):
    """Every stage from what the one before gave on the GPU, against the definition in 64 bits."""
    import torch

    print("layer", t, padded, flush=True)
    layer = Layer(wq)
    x, res = _inputs(t, t)
    real = torch.arange(t, device="cuda") < (t + 1) // 2 if padded else None
    o = layer(x, res, real)
    stream = (x.float() + res.float()).to(torch.bfloat16)
    assert torch.equal(o["stream"], stream)
    f = lambda a: a.double().cpu().numpy()
    codes, a = i8.quantize(f(stream) * f(layer.norm))
    assert np.array_equal(o["rows"].codes.cpu().numpy(), codes)
    scales = o["rows"].scales.cpu().numpy()
    _, inv = i8.norm(f(stream), f(layer.norm), 1e-6)
    i8.assert_within(scales, a * inv[:, 0] / 127, a * inv[:, 0] / 127 * (i8.additions(HIDDEN) + 8) * i8.U, "scales")
    rc, rs = _weight(layer.router)
    assert np.array_equal(f(o["logits"]), i8.product_bits(codes, scales, rc[0], rs[0], "f32"))
    ids = o["ids"].cpu().numpy()
    loss, bound, counts, d_logits, bd = i8.balance_bounds(f(o["logits"]), ids, 0.01, "f32")
    assert np.array_equal(o["counts"].cpu().numpy(), counts)
    i8.assert_within(o["loss"].item(), loss, bound, "loss")
    i8.assert_within(f(o["d_logits"]), d_logits, bd, "d_logits")
    offsets, order, positions = mx.route(ids, E)
    assert np.array_equal(o["offsets"].cpu().numpy(), offsets) and np.array_equal(o["positions"].cpu().numpy(), positions)
    (gc, gs), (uc, us), (dc, dsc) = (_weight(w) for w in (layer.gate, layer.up, layer.down))
    h, d = f(o["h"]), f(o["d"])
    hc, hs = o["hq"].codes.cpu().numpy(), o["hq"].scales.cpu().numpy()
    want, a = i8.quantize(h)
    assert np.array_equal(hc, want) and np.array_equal(hs, i8.f32(a / 127))
    for e in range(E):
        at = slice(offsets[e], offsets[e + 1])
        tok = order[at] // TOPK
        ref, bound = i8.gate_up_bound(codes[tok], scales[tok], gc[e], gs[e], uc[e], us[e])
        i8.assert_within(h[at], ref, bound, f"h of expert {e}")
        assert np.array_equal(d[at], i8.product_bits(hc[at], hs[at], dc[e], dsc[e], "f32")), e
    w = f(o["weights"])
    used = positions >= 0
    picked = np.where(used[:, :, None], d[np.where(used, positions, 0)], 0.0)
    ref, mags = (w[:, :, None] * picked).sum(1), np.abs(w[:, :, None] * picked).sum(1)
    i8.assert_within(f(o["y"]), ref, (TOPK + 1) * i8.U * mags + 2.0 ** -140, "y")
    if padded:
        assert (o["y"][(t + 1) // 2:] == 0).all() and (o["d_logits"][(t + 1) // 2:] == 0).all()


@pytest.mark.parametrize("t", [1, 40, 700])
def test_layer_captured(wq, t):
    """One graph of the layer, replayed over new inputs with eager work between the replays."""
    import torch

    print("captured", t, flush=True)
    layer = Layer(wq, 1)
    x, res = _inputs(t, 1)
    keep = ("rows", "stream", "loss", "counts", "h", "d", "y", "d_logits")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer(x, res)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(x, res)
    for i in range(4):
        a, b = _inputs(t, 50 + i)
        want = layer(a, b)
        x.copy_(a)
        res.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        for k in keep:
            g, w = (out[k].codes, want[k].codes) if k == "rows" else (out[k], want[k])
            assert torch.equal(g, w), (i, k)


def test_gradients_captured(wq):
    import torch

    for n, k, dt in ((3, 64, torch.bfloat16), (700, 1111, torch.float32)):
        x, ds, dy = (torch.randn((n, k), device="cuda").to(dt) for _ in range(3))
        w = torch.randn(k, device="cuda").to(dt)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            wq.wq_rms_norm_grad(dy, x, w, ds)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = wq.wq_rms_norm_grad(dy, x, w, ds)
        for i in range(3):
            dy.copy_(torch.randn((n, k), device="cuda"))
            want = wq.wq_rms_norm_grad(dy, x, w, ds)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1]), i


def test_two_streams(wq):
    """The same calls on two streams at once, each with workspaces of its own, give what one gives alone."""
    import torch

    layer = Layer(wq, 2)
    inputs = [_inputs(700, 7), _inputs(300, 8)]
    want = [layer(*i) for i in inputs]
    grads = [wq.wq_rms_norm_grad(i[0], w["stream"], layer.norm, i[1]) for i, w in zip(inputs, want)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got, got_grads = [[], []], [[], []]
    for _ in range(5):
        for n, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[n].append(layer(*inputs[n]))
                got_grads[n].append(wq.wq_rms_norm_grad(inputs[n][0], want[n]["stream"], layer.norm, inputs[n][1]))
    torch.cuda.synchronize()
    for n in range(2):
        for o, g in zip(got[n], got_grads[n]):
            assert all(torch.equal(o[k], want[n][k]) for k in ("stream", "loss", "counts", "h", "d", "y", "d_logits"))
            assert torch.equal(g[0], grads[n][0]) and torch.equal(g[1], grads[n][1])


def test_training_step(wq):
    """Norm with residual and router with balance loss in autograd functions: every gradient against torch's
    autograd of the definitions in 64 bits."""
    import torch

    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, residual, weight):
            y, total = wq.wq_rms_norm(x, weight, residual, eps=1e-5)
            ctx.save_for_backward(total, weight)
            return y, total

        @staticmethod
        def backward(ctx, dy, d_sum):
            total, weight = ctx.saved_tensors
            dx, dw = wq.wq_rms_norm_grad(dy.contiguous(), total, weight, d_sum.contiguous(), eps=1e-5)
            return dx, dx, dw

    class Balance(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, ids):
            loss, counts = wq.wq_moe_balance_loss(logits, ids, 0.5)
            ctx.save_for_backward(logits, ids, counts)
            return loss

        @staticmethod
        def backward(ctx, d_loss):
            logits, ids, counts = ctx.saved_tensors
            return wq.wq_moe_balance_loss_grad(logits, ids, counts, 0.5, d_loss), None

    t, k = 65, 100
    g = torch.Generator().manual_seed(3)
    x, res, c, u = (torch.randn((t, k), generator=g) for _ in range(4))
    weight = 1 + 0.2 * torch.randn(k, generator=g)
    router = torch.randn((E, k), generator=g) * 0.2
    ids = torch.topk(torch.randn((t, E), generator=g), TOPK, dim=1).indices.to(torch.int32)
    ids[60:] = -1

    def leaves(dtype, device):
        return [v.to(dtype=dtype, device=device).requires_grad_() for v in (x, res, weight, router)]

    a = leaves(torch.float32, "cuda")
    y, total = Norm.apply(a[0], a[1], a[2])
    loss = (y * c.cuda()).sum() + (total * u.cuda()).sum() + Balance.apply(y @ a[3].t(), ids.cuda())
    loss.backward()
    b = leaves(torch.float64, "cpu")
    r = b[0] + b[1]
    y = r * torch.rsqrt((r * r).mean(1, keepdim=True) + 1e-5) * b[2]
    p = torch.softmax(y @ b[3].t(), 1)[:60]
    share = E * torch.bincount(ids[:60].reshape(-1).long(), minlength=E) / (60 * TOPK)
    ref = (y * c).sum() + (r * u).sum() + 0.5 * (share * p.mean(0)).sum()
    ref.backward()
    # fp32 throughout: sums of up to 100 x 65 terms, each off by a few 2^-24 of magnitudes near one
    assert abs(loss.item() - ref.item()) < 1e-3
    for got, want in zip(a, b):
        d = got.grad.double().cpu() - want.grad
        assert d.abs().max() <= 2e-5 * want.grad.abs().max(), d.abs().max()


def test_int8_rows_of_the_norm_are_those_of_the_quantiser(wq):
    """wq_rms_norm_i8 of bf16 rows with a weight of ones gives the codes of wq_quantize_i8 of the rows."""
    import torch

    x = torch.randn((50, 1111), device="cuda").to(torch.bfloat16)
    rows, _ = wq.wq_rms_norm_i8(x, torch.ones(1111, device="cuda", dtype=torch.bfloat16))
    assert torch.equal(rows.codes, wq.wq_quantize_i8(x).codes)
