"""The root-mean-square norm with the residual's addition, in its own type and in int8, and its gradients, on
the GPU against the definitions in 64 bits (i8_testutil)."""
import sys

import numpy as np
import pytest

import i8_testutil as i8

pytestmark = pytest.mark.gpu

EPS = 1e-6
# one element, shorter than a piece, a quarter wave's rows, one wave's with and without a ragged end, several
# waves', and rows that are read again (from 65537 bf16 or 32769 fp32 values on)
LENGTHS = [1, 5, 8, 64, 136, 513, 1024, 1111, 2048, 4096, 4099, 8192, 12000, 16384, 20001, 40000, 66000, 70003]
# few rows, and (where that takes other kernels) more than there are CUs
ROWS = [(5, k) for k in LENGTHS] + [(300, k) for k in (40, 136, 513, 700, 1111, 2048, 3001, 4099, 8192, 12000)]


@pytest.fixture(scope="module")
def wq():
    import torch

    import weight_only_bit_amd as wq

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    wq.lib()
    return wq


def _dtype(name):
    import torch

    return torch.bfloat16 if name == "bf16" else torch.float32


def _inputs(n, k, dtype, seed=0):
    import torch

    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, k, generator=g)
    res = torch.randn(n, k, generator=g) * 3
    w = 1 + 0.3 * torch.randn(k, generator=g)
    return [t.to(_dtype(dtype)) for t in (x, res, w)]


def _stored(x, res):
    """The sum as it is stored: fp32 addition (exact, or its own rounding), one rounding to the type."""
    return (x.float() + res.float()).to(x.dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,k", ROWS)
def test_norm(wq, dtype, n, k):
    import torch

    print("norm", dtype, n, k, flush=True)
    x, res, w = _inputs(n, k, dtype, k)
    r = _stored(x, res)
    y, total = wq.wq_rms_norm(x.cuda(), w.cuda(), res.cuda(), eps=EPS)
    assert torch.equal(total.cpu(), r)
    i8.assert_within(i8.to_host(y), *i8.norm_bound(r.double().numpy(), w.double().numpy(), EPS, dtype), "y")
    # without a residual
    xc = x.cuda()
    y, total = wq.wq_rms_norm(xc, w.cuda(), eps=EPS)
    assert total is xc
    i8.assert_within(i8.to_host(y), *i8.norm_bound(x.double().numpy(), w.double().numpy(), EPS, dtype), "y alone")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,k", ROWS)
def test_norm_i8(wq, dtype, n, k):
    import torch

    print("norm i8", dtype, n, k, flush=True)
    x, res, w = _inputs(n, k, dtype, k + 1)
    r = _stored(x, res)
    rows, total = wq.wq_rms_norm_i8(x.cuda(), w.cuda(), res.cuda(), eps=EPS)
    assert torch.equal(total.cpu(), r)
    rd, wd = r.double().numpy(), w.double().numpy()
    codes, a = i8.quantize(rd * wd)
    assert np.array_equal(rows.codes.cpu().numpy(), codes)
    _, inv = i8.norm(rd, wd, EPS)
    ref = a * inv[:, 0] / 127
    rel = ((i8.additions(k) + 2) / 2 + 6) * i8.U
    i8.assert_within(i8.to_host(rows.scales), ref, ref * rel + 2.0 ** -140, "scales")
    alone, _ = wq.wq_rms_norm_i8(r.cuda(), w.cuda(), eps=EPS)
    assert torch.equal(alone.codes, rows.codes) and torch.equal(alone.scales, rows.scales)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k", [8, 1111, 8192, 70003])
def test_sum_in_place(wq, dtype, k):
    """The sum may take x's or the residual's place, also where a row's end is ragged."""
    import torch

    print("in place", dtype, k, flush=True)
    x, res, w = (t.cuda() for t in _inputs(6, k, dtype, 3))
    y, total = wq.wq_rms_norm(x, w, res)
    rows, _ = wq.wq_rms_norm_i8(x, w, res)
    for which in ("x", "residual"):
        a, b = x.clone(), res.clone()
        into = a if which == "x" else b
        y2, t2 = wq.wq_rms_norm(a, w, b, sum=into)
        assert t2 is into and torch.equal(t2, total) and torch.equal(y2, y), which
        a, b = x.clone(), res.clone()
        into = a if which == "x" else b
        rows2, t2 = wq.wq_rms_norm_i8(a, w, b, sum=into)
        assert torch.equal(t2, total) and torch.equal(rows2.codes, rows.codes) and torch.equal(rows2.scales, rows.scales)
    # x and the residual one tensor
    a = x.clone()
    y3, t3 = wq.wq_rms_norm(a, w, a, sum=a)
    assert t3 is a and torch.equal(a, _stored(x, x))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_edges(wq, dtype):
    """Rows of zeros, of tiny and of huge values, infinities and NaN; no row touches another."""
    import torch

    x = torch.randn(8, 100).to(_dtype(dtype))
    x[0] = 0
    x[1] *= 1e-20
    x[2] *= 1e18
    x[3, 7] = float("inf")
    x[4, 99] = float("nan")
    w = torch.ones(100, dtype=x.dtype)
    y, _ = wq.wq_rms_norm(x.cuda(), w.cuda(), eps=EPS)
    y = y.cpu()
    assert (y[0] == 0).all() and y[4].isnan().all() and y[3, 7].isnan()
    ok = [0, 1, 2, 5, 6, 7]
    i8.assert_within(y[ok].double().numpy(), *i8.norm_bound(x[ok].double().numpy(), w.double().numpy(), EPS, dtype), "y")
    rows, _ = wq.wq_rms_norm_i8(x.cuda(), w.cuda(), eps=EPS)
    codes, scales = rows.codes.cpu(), rows.scales.cpu()
    assert (codes[[0, 3, 4]] == 0).all() and scales[0] == 0 and scales[3].isnan() and scales[4].isnan()
    assert np.array_equal(codes.numpy()[ok], i8.quantize(x[ok].double().numpy())[0])
    assert scales[ok].isfinite().all()
    # an infinite weight meets every row
    w[3] = float("inf")
    rows, _ = wq.wq_rms_norm_i8(x.cuda(), w.cuda(), eps=EPS)
    assert rows.scales.isnan().all() and (rows.codes == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,k", [(1, 1), (3, 5), (1, 8192), (700, 64), (2100, 100), (513, 1024), (33, 1111), (700, 2050),
                                 (40, 4096), (300, 700), (300, 3001), (600, 8192), (257, 12000), (9, 16390), (30, 40000), (5, 70003), (520, 33000)])
def test_gradients(wq, dtype, n, k):
    print("gradients", dtype, n, k, flush=True)
    x, res, w = _inputs(n, k, dtype, 5)
    dy, ds, _ = _inputs(n, k, dtype, 6)
    r = _stored(x, res)
    dx, dw = wq.wq_rms_norm_grad(dy.cuda(), r.cuda(), w.cuda(), ds.cuda(), eps=EPS)
    f = lambda t: t.double().numpy()
    rx, bx, rw, bw = i8.norm_grad_bounds(f(dy), f(r), f(w), EPS, f(ds), dtype)
    i8.assert_within(i8.to_host(dx), rx, bx, "dx")
    i8.assert_within(i8.to_host(dw), rw, bw, "d_weight")
    # without the sum's own gradient, and without the weight's
    dx0, none = wq.wq_rms_norm_grad(dy.cuda(), r.cuda(), w.cuda(), eps=EPS, weight_grad=False)
    assert none is None
    rx, bx, _, _ = i8.norm_grad_bounds(f(dy), f(r), f(w), EPS, 0.0 * f(ds), dtype)
    i8.assert_within(i8.to_host(dx0), rx, bx, "dx alone")


def test_gradients_in_place_and_empty(wq):
    import torch

    for dtype, k in (("bf16", 1111), ("f32", 70003)):
        x, ds, w = (t.cuda() for t in _inputs(40, k, dtype, 8))
        dy = torch.randn_like(x)
        dx, dw = wq.wq_rms_norm_grad(dy, x, w, ds)
        into = ds.clone()
        dx2, dw2 = wq.wq_rms_norm_grad(dy, x, w, into, dx=into)
        assert dx2 is into and torch.equal(dx2, dx) and torch.equal(dw2, dw)
        e = x[:0]
        dx0, dw0 = wq.wq_rms_norm_grad(e, e, w, d_weight=torch.ones(k, device="cuda"))
        assert dx0.shape == (0, k) and (dw0 == 0).all()
        y, total = wq.wq_rms_norm(e, w, e)
        assert y.shape == total.shape == (0, k)


def test_gradient_against_differences(wq):
    """The kernel's gradients along random directions against central differences of the 64-bit norm."""
    rng = np.random.default_rng(1)
    n, k, h = 7, 1111, 1e-5
    x, ds, w = _inputs(n, k, "f32", 9)
    dy = _inputs(n, k, "f32", 10)[0]
    dx, dw = wq.wq_rms_norm_grad(dy.cuda(), x.cuda(), w.cuda(), ds.cuda(), eps=1e-3)
    f = lambda r, v: (i8.norm(r, v, 1e-3)[0] * dy.double().numpy()).sum() + (r * ds.double().numpy()).sum()
    r, v = x.double().numpy(), w.double().numpy()
    for _ in range(4):
        u, s = rng.standard_normal((n, k)), rng.standard_normal(k)
        got = (i8.to_host(dx) * u).sum()
        # the differences' own error, and fp32's in the kernel: below 1e-5 of the terms' magnitudes
        assert abs((f(r + h * u, v) - f(r - h * u, v)) / (2 * h) - got) < 1e-5 * (np.abs(i8.to_host(dx) * u)).sum()
        got = (i8.to_host(dw) * s).sum()
        assert abs((f(r, v + h * s) - f(r, v - h * s)) / (2 * h) - got) < 1e-5 * np.abs(i8.to_host(dw) * s).sum()


def test_many_rows(wq):
    """More rows than workgroups of a launch hold at a time, each as the same row alone; gradients repeat."""
    import torch

    x = torch.randn(70001, 40, device="cuda").to(torch.bfloat16)
    w = torch.randn(40, device="cuda").to(torch.bfloat16)
    y, _ = wq.wq_rms_norm(x, w, x)
    some = torch.arange(0, 70001, 3001)
    y2, _ = wq.wq_rms_norm(x[some], w, x[some])
    assert torch.equal(y[some], y2)
    first = wq.wq_rms_norm_grad(y, x, w, x)
    for _ in range(2):
        again = wq.wq_rms_norm_grad(y, x, w, x)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_rows_beyond_32_bits(wq):
    """Rows beyond 2^31 elements."""
    import torch

    print("beyond 32 bits", flush=True)
    n, k = 270000, 8192
    x = torch.randn(n, k, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(k, device="cuda").to(torch.bfloat16)
    rows, total = wq.wq_rms_norm_i8(x, w, x)
    tail, t2 = wq.wq_rms_norm_i8(x[-5:].clone(), w, x[-5:].clone())
    assert torch.equal(rows.codes[-5:], tail.codes) and torch.equal(rows.scales[-5:], tail.scales)
    assert torch.equal(total[-5:], t2)
    del rows
    y, _ = wq.wq_rms_norm(x, w)
    dx, _ = wq.wq_rms_norm_grad(y, x, w, total)
    d2, _ = wq.wq_rms_norm_grad(y[-5:].clone(), x[-5:].clone(), w, total[-5:].clone())
    assert torch.equal(dx[-5:], d2)


def test_columns_beyond_one_launch(wq):
    """Two rows of more than 2^28 values: the weight's gradient takes several launches."""
    import torch

    print("columns beyond one launch", flush=True)
    k = (1 << 28) + 72
    x = torch.randn((2, 1 << 20), device="cuda").to(torch.bfloat16).repeat(1, k // (1 << 20) + 1)[:, :k].contiguous()
    dy = torch.roll(x, 1, 0)
    w = torch.ones(k, device="cuda", dtype=torch.bfloat16)
    dx, dw = wq.wq_rms_norm_grad(dy, x, w)
    inv = [1 / (x[i].double().square().mean() + EPS).sqrt().item() for i in range(2)]
    for at in (0, k // 2, k - 64):
        s = slice(at, at + 64)
        ref = sum(dy[i, s].double() * x[i, s].double() * inv[i] for i in range(2))
        mags = sum((dy[i, s].double() * x[i, s].double() * inv[i]).abs() for i in range(2))
        # the mean's chain of additions is k / 1024 long
        assert ((dw[s].double() - ref).abs() <= (i8.additions(k) + 20) * i8.U * mags + 1e-30).all()
