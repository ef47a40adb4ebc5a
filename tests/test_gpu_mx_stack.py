"""MXFP4 experts in the framework's own paths: layers of a MoeStack beside INT4 ones, captured and
replayed, and the FFN without a caller's workspace.  Both run the same stages as wq_moe_ffn (itself
tested against 64 bits), so they give the same bits."""
import numpy as np
import pytest

import mx_testutil as mx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [1, 24, 300])
def test_stack_and_noalloc(t):
    import torch

    import weight_only_bit_amd as wq
    from weight_only_bit_amd.stack import MoeStack

    E, inter, hidden, topk = 8, 192, 320, 4
    print("stack", t, flush=True)
    rng = np.random.default_rng(t)

    def mxfp4():
        return tuple(mx.weight(wq, *mx.random_codes(rng, E, *s)) for s in ((inter, hidden), (inter, hidden), (hidden, inter)))

    def int4():
        out = []
        for n, k in ((inter, hidden), (inter, hidden), (hidden, inter)):
            codes = torch.from_numpy(rng.integers(0, 256, (E, n, k // 2)).astype(np.uint8)).cuda()
            scales = (torch.rand((E, n, k // 64), device="cuda") * 0.01 + 0.01).to(torch.bfloat16)
            out.append(wq.PackedWeight(wq.FMT_INT4, n, k, E, 64, codes=codes, scales=scales, zp=8))
        return tuple(out)

    layers = [mxfp4(), int4(), mxfp4()]
    x = torch.from_numpy(rng.standard_normal((t, hidden))).to(torch.bfloat16).cuda()
    routes, ys = [], []
    for _ in layers:
        ids = np.argsort(rng.random((t, E)), 1)[:, :topk].astype(np.int32)
        routes.append((torch.from_numpy(ids).cuda(), torch.from_numpy(rng.random((t, topk)).astype(np.float32)).cuda()))
        ys.append(torch.empty((t, hidden), dtype=torch.bfloat16, device="cuda"))
    want = [wq.wq_moe_ffn(x, *r, *l) for l, r in zip(layers, routes)]
    for l, r, w in zip(layers, routes, want):
        y = torch.empty_like(w)
        assert torch.equal(wq.wq_moe_ffn_noalloc(x, *r, *l, y), w)
    stack = MoeStack(layers, t, topk)
    stack.step(x, routes, ys)
    for y, w in zip(ys, want):
        assert torch.equal(y, w)
    stack.capture(x, routes, ys)
    for i in range(3):
        x.copy_(torch.from_numpy(rng.standard_normal((t, hidden))).to(torch.bfloat16))
        want = [wq.wq_moe_ffn(x, *r, *l) for l, r in zip(layers, routes)]
        torch.cuda.synchronize()
        for y in ys:
            y.zero_()
        stack.replay()
        torch.cuda.synchronize()
        for y, w in zip(ys, want):
            assert torch.equal(y, w), i
