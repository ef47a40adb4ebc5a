"""Token dispatch on the GPU (positions, permutation, the weighted way back, gradients) against
plain numpy in 64 bits.

Tolerances: a permuted row is a copy (exact).  A sum of topk weighted values is at most 2 topk fp32
roundings of partial sums below the sum of magnitudes, then one rounding to the type: the bound of
mx_testutil.sum_bound with K = 2 topk.  w * dy is one rounding in fp32 and one to the type; a dot
product over hidden values is that bound with K = 2 hidden."""
import sys

import numpy as np
import pytest

import mx_testutil as mx

pytestmark = pytest.mark.gpu


def _say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def wq():
    import torch

    import weight_only_bit_amd as wq

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    wq.lib()
    return wq


def _type(name):
    import torch

    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _rand(rng, dtype, *shape):
    x = rng.standard_normal(shape)
    return mx.bf16(x) if dtype == "bf16" else x.astype(np.float32).astype(np.float64)


def _cuda(a, dtype=None):
    import torch

    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def _plan(rng, t, topk, E, dropped):
    ids = rng.integers(0, E, (t, topk)).astype(np.int32)
    if dropped:
        ids[rng.random((t, topk)) < 0.25] = -1
        ids[rng.random((t, topk)) < 0.1] = E + 3
        ids[t // 2] = E  # one token loses every pair
    return ids, *mx.route(ids, E)


@pytest.mark.parametrize("t,topk,E,dropped", [(1, 1, 1, False), (1, 8, 512, False), (5, 3, 4, True), (300, 8, 64, True),
                                             (1025, 4, 7, False), (1, 2, 4, True)])
def test_positions(wq, t, topk, E, dropped):
    _say("positions", t, topk, E, dropped)
    ids, off, order, pos = _plan(np.random.default_rng(t), t, topk, E, dropped)
    offsets, pairs = wq.wq_moe_route(_cuda(ids), E)
    got = wq.wq_moe_positions(_cuda(ids), offsets, pairs)
    assert got.shape == (t, topk) and np.array_equal(got.cpu().numpy(), pos)


SIZES = [(1, 1, 1, 1), (3, 2, 4, 7), (40, 8, 64, 64), (40, 8, 64, 100), (17, 3, 5, 257), (33, 9, 16, 1027), (64, 17, 32, 320),
         (9, 2, 3, 8192), (300, 4, 8, 2049), (5, 1, 2, 8), (6, 5, 4, 33)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dropped", [False, True])
@pytest.mark.parametrize("t,topk,E,hidden", SIZES)
def test_forward(wq, t, topk, E, hidden, dropped, dtype):
    import torch

    _say("dispatch", t, topk, E, hidden, dropped, dtype)
    rng = np.random.default_rng(t * hidden)
    ids, off, order, pos = _plan(rng, t, topk, E, dropped)
    positions = _cuda(pos)
    x = _rand(rng, dtype, t, hidden)
    P, dt = t * topk, _type(dtype)
    rows = torch.full((P, hidden), 5.0, dtype=dt, device="cuda")
    got = mx.to_host(wq.wq_moe_permute(_cuda(x, dt), positions, rows=rows))
    assert np.array_equal(got[:len(order)], x[order // topk])
    assert np.all(got[len(order):] == 5.0)
    # back: rows of no pair hold NaN, which no sum may take in
    r = _rand(rng, dtype, P, hidden)
    r[len(order):] = np.nan
    wts = rng.standard_normal((t, topk)).astype(np.float32)
    wts[pos < 0] = np.nan
    safe = np.where((pos >= 0)[:, :, None], np.nan_to_num(r)[np.maximum(pos, 0)], 0.0)
    for w in (None, wts):
        w64 = (np.ones((t, topk)) if w is None else np.nan_to_num(w.astype(np.float64)))[:, :, None]
        ref, mag = (w64 * safe).sum(1), np.abs(w64 * safe).sum(1)
        y = wq.wq_moe_unpermute(_cuda(r, dt), positions, None if w is None else _cuda(w))
        mx.assert_within(mx.to_host(y), ref, mx.sum_bound(ref, mag, 2 * topk, dtype), "unpermute")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dropped", [False, True])
@pytest.mark.parametrize("t,topk,E,hidden", SIZES)
def test_gradients(wq, t, topk, E, hidden, dropped, dtype):
    import torch

    _say("dispatch grad", t, topk, E, hidden, dropped, dtype)
    rng = np.random.default_rng(t + hidden)
    ids, off, order, pos = _plan(rng, t, topk, E, dropped)
    positions, dt, P = _cuda(pos), _type(dtype), t * topk
    dy, r = _rand(rng, dtype, t, hidden), _rand(rng, dtype, P, hidden)
    wts = rng.standard_normal((t, topk)).astype(np.float32)
    for w in (wts, None):
        w64 = np.ones((t, topk)) if w is None else w.astype(np.float64)
        out = torch.full((P, hidden), 5.0, dtype=dt, device="cuda")
        d_rows, d_w = wq.wq_moe_unpermute_grad(_cuda(dy, dt), _cuda(r, dt), positions,
                                               None if w is None else _cuda(w), d_rows=out)
        got = mx.to_host(d_rows)
        ref = w64.reshape(-1)[order][:, None] * dy[order // topk]
        mx.assert_within(got[:len(order)], ref, mx.sum_bound(ref, np.abs(ref), 1, dtype), "d_rows")
        assert np.all(got[len(order):] == 5.0)
        safe = np.where((pos >= 0)[:, :, None], r[np.maximum(pos, 0)], 0.0)
        ref, mag = (safe * dy[:, None]).sum(2), np.abs(safe * dy[:, None]).sum(2)
        mx.assert_within(mx.to_host(d_w), ref, mx.sum_bound(ref, mag, 2 * hidden, "f32"), "d_weights")
    # the gradient of the permutation: every token's sum over its rows
    dx = wq.wq_moe_unpermute(_cuda(r, dt), positions)
    ref, mag = safe.sum(1), np.abs(safe).sum(1)
    mx.assert_within(mx.to_host(dx), ref, mx.sum_bound(ref, mag, 2 * topk, dtype), "dx")
    only, none = wq.wq_moe_unpermute_grad(_cuda(dy, dt), None, positions, _cuda(wts), d_rows=torch.full_like(out, 5.0))
    assert none is None
    again, _ = wq.wq_moe_unpermute_grad(_cuda(dy, dt), _cuda(r, dt), positions, _cuda(wts), d_rows=torch.full_like(out, 5.0))
    assert torch.equal(only, again)


def test_gradients_against_differences(wq):
    """The operators are linear in the rows and in the weights, so a difference over any step is
    the gradient's product with it, up to the roundings of its two fp32 values."""
    import torch

    rng = np.random.default_rng(7)
    t, topk, E, hidden = 11, 3, 4, 130
    ids, off, order, pos = _plan(rng, t, topk, E, True)
    positions = _cuda(pos)
    rows, step = (torch.from_numpy(rng.standard_normal((t * topk, hidden))).float().cuda() for _ in range(2))
    w, wstep = (torch.from_numpy(rng.standard_normal((t, topk))).float().cuda() for _ in range(2))
    dy = torch.from_numpy(rng.standard_normal((t, hidden))).float().cuda()
    d_rows, d_w = wq.wq_moe_unpermute_grad(dy, rows, positions, w, d_rows=torch.zeros_like(rows))
    y0 = wq.wq_moe_unpermute(rows, positions, w).double()
    for got, want in (((wq.wq_moe_unpermute(rows + step, positions, w).double() - y0), (d_rows, step)),
                      ((wq.wq_moe_unpermute(rows, positions, w + wstep).double() - y0), (d_w, wstep))):
        lhs = float((got * dy.double()).sum())
        rhs = float((want[0].double() * want[1].double()).sum())
        # y values are sums of topk products below 6 * 6 each, dy below 6, t * hidden of them
        assert abs(lhs - rhs) <= t * hidden * 6 * (2 * topk) * (topk * 36) * 2.0 ** -23, (lhs, rhs)


def test_dispatch_in_training(wq):
    """route -> positions -> permute -> the experts' matrices -> back, and all gradients, as a
    training step around frozen experts runs them, against autograd in 64 bits."""
    import torch

    rng = np.random.default_rng(8)
    t, topk, E, hidden = 50, 2, 4, 96
    ids, off, order, pos = _plan(rng, t, topk, E, True)
    x, w = rng.standard_normal((t, hidden)), rng.random((t, topk))
    mats = rng.standard_normal((E, hidden, hidden)) / hidden ** 0.5
    dy = rng.standard_normal((t, hidden))
    x32, w32, m32, dy32 = (torch.from_numpy(a).float() for a in (x, w, mats, dy))
    offsets, pairs = wq.wq_moe_route(_cuda(ids), E)
    positions = wq.wq_moe_positions(_cuda(ids), offsets, pairs)
    at = offsets.tolist()
    rows = wq.wq_moe_permute(x32.cuda(), positions, rows=torch.zeros((t * topk, hidden), device="cuda"))
    z = torch.zeros_like(rows)
    mg = m32.cuda()
    for e in range(E):
        z[at[e]:at[e + 1]] = rows[at[e]:at[e + 1]] @ mg[e].t().contiguous()
    y = wq.wq_moe_unpermute(z, positions, w32.cuda())
    dz, dw = wq.wq_moe_unpermute_grad(dy32.cuda(), z, positions, w32.cuda(), d_rows=torch.zeros_like(z))
    dr = torch.zeros_like(rows)
    for e in range(E):
        dr[at[e]:at[e + 1]] = dz[at[e]:at[e + 1]] @ mg[e]
    dx = wq.wq_moe_unpermute(dr, positions)
    xa, wa = x32.double().requires_grad_(), w32.double().requires_grad_()
    ya = torch.zeros(t, hidden, dtype=torch.float64)
    for j in range(topk):
        e = torch.from_numpy(ids[:, j].astype(np.int64))
        ok = ((e >= 0) & (e < E)).double()
        mj = m32.double()[e.clamp(0, E - 1)]
        ya = ya + ((wa[:, j] * ok)[:, None] * (mj @ xa[:, :, None])[:, :, 0])
    (ya * dy32.double()).sum().backward()
    for got, ref in ((y, ya.detach()), (dx, xa.grad), (dw, wa.grad)):
        # three fp32 sums of at most hidden terms one after another, values of order 1
        np.testing.assert_allclose(mx.to_host(got), ref.numpy(), rtol=0, atol=3 * hidden * 2.0 ** -23 * 30)


def test_dispatch_captured(wq):
    import torch

    rng = np.random.default_rng(6)
    t, topk, E, hidden = 90, 4, 8, 264
    new = lambda: (_cuda(_plan(rng, t, topk, E, True)[0]), torch.randn(t, hidden, device="cuda").bfloat16(),
                   torch.rand(t, topk, device="cuda"), torch.randn(t, hidden, device="cuda").bfloat16())
    rows = torch.zeros((t * topk, hidden), dtype=torch.bfloat16, device="cuda")
    d_rows = torch.zeros_like(rows)

    def run(a):
        ids, x, w, dy = a
        offsets, pairs = wq.wq_moe_route(ids, E)
        positions = wq.wq_moe_positions(ids, offsets, pairs)
        rows.zero_()
        d_rows.zero_()
        r = wq.wq_moe_permute(x, positions, rows=rows)
        y = wq.wq_moe_unpermute(r, positions, w)
        dr, dw = wq.wq_moe_unpermute_grad(dy, r, positions, w, d_rows=d_rows)
        return y, dw, wq.wq_moe_unpermute(dr, positions)

    live = new()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(live)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = run(live)
    for _ in range(4):
        other = new()
        want = [o.clone() for o in run(other)]
        for a, b in zip(live, other):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        for o, v in zip(outs, want):
            assert torch.equal(o, v)


def test_refusals(wq):
    import torch

    pos = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    x = torch.randn(4, 64, device="cuda")
    rows = torch.randn(8, 64, device="cuda")
    with pytest.raises(TypeError, match="dtype"):
        wq.wq_moe_permute(x, pos.long())
    with pytest.raises(ValueError, match="positions must be"):
        wq.wq_moe_permute(x, pos.view(-1))
    with pytest.raises(ValueError, match="shape"):
        wq.wq_moe_permute(x[:3], pos)
    with pytest.raises(TypeError, match="dtype"):
        wq.wq_moe_permute(x, pos, rows=rows.bfloat16())
    with pytest.raises(TypeError, match="neither"):
        wq.wq_moe_unpermute(rows.half(), pos)
    with pytest.raises(ValueError, match="shape"):
        wq.wq_moe_unpermute(rows, pos, torch.ones(4, 3, device="cuda"))
    with pytest.raises(TypeError, match="f32"):
        wq.wq_moe_unpermute(rows, pos, torch.ones(4, 2, device="cuda").bfloat16())
    with pytest.raises(ValueError, match="contiguous"):
        wq.wq_moe_unpermute(torch.randn(64, 8, device="cuda").t(), pos)
    with pytest.raises(TypeError, match="dtype"):
        wq.wq_moe_unpermute_grad(x, rows.bfloat16(), pos)
    with pytest.raises(ValueError, match="WQ_ERR_ALIGN"):
        wq.wq_moe_permute(torch.randn(4 * 64 + 1, device="cuda")[1:].view(4, 64), pos)
    with pytest.raises(ValueError, match="elements"):
        wq.wq_moe_positions(pos, torch.zeros(5, dtype=torch.int32, device="cuda"), torch.zeros(7, dtype=torch.int32, device="cuda"))
