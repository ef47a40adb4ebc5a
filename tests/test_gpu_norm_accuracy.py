"""Digits of the norm's weight gradient, and rows of zeros without an epsilon, on the GPU against the definitions in
64 bits."""
import numpy as np
import pytest

import i8_testutil as i8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wq():
    import torch

    import weight_only_bit_amd as wq

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    wq.lib()
    return wq


# rows that share a workgroup and rows of one each; at most one row a lane
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,k", [(4096, 40), (1600, 500), (336, 1111), (256, 8192), (64, 33000)])
def test_large_rows_leave_the_weights_small_gradients(wq, dtype, n, k):
    """The first 16 rows' gradients are 2^20 and those of the last 16 the same with the other sign, so their terms
    cancel bit for bit between the workgroups; what the rows between them add keeps its digits: a term's roundings
    (inv's chain among them) and the 16 rows' that meet in a workgroup, of these rows' magnitudes."""
    import torch

    print("large rows", dtype, n, k, flush=True)
    rng = np.random.default_rng(k)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    row = torch.from_numpy(rng.standard_normal(k)).to(dt)
    r = row.repeat(n, 1)
    dy = torch.from_numpy(rng.standard_normal((n, k))).to(dt)
    dy[:16], dy[n - 16:] = 2.0 ** 20, -2.0 ** 20
    _, dw = wq.wq_rms_norm_grad(dy.cuda(), r.cuda(), torch.ones(k, dtype=dt).cuda(), eps=1e-6)
    f = lambda t: t.double().numpy()
    inv = 1 / np.sqrt((f(row) ** 2).mean() + 1e-6)
    terms = f(dy)[16: n - 16] * f(row) * inv
    i8.assert_within(i8.to_host(dw), terms.sum(0), (i8.additions(k) + 5 + 16 + 1) * i8.U * np.abs(terms).sum(0), "d_weight")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k", [5, 64, 1111, 8192, 70003])
def test_rows_of_zeros_without_an_epsilon(wq, dtype, k):
    """eps = 0: a row of zeros, or of values whose squares vanish, is normed to zeros (scale 0 in int8) and passes no
    gradient on but the sum's own; the rows beside it, a NaN's too, are as ever."""
    import torch

    print("no epsilon", dtype, k, flush=True)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    g = torch.Generator().manual_seed(k)
    x, dy, ds = (torch.randn((9, k), generator=g).to(dt) for _ in range(3))
    w = (1 + 0.1 * torch.randn(k, generator=g)).to(dt)
    x[2], x[5] = 0, 1e-30
    x[7, k // 2] = float("nan")
    ok = [0, 1, 3, 4, 6, 8]
    f = lambda t: t.double().numpy()
    y, _ = wq.wq_rms_norm(x.cuda(), w.cuda(), eps=0.0)
    y = y.cpu()
    assert (y[[2, 5]] == 0).all() and y[7].isnan().all()
    i8.assert_within(f(y[ok]), *i8.norm_bound(f(x[ok]), f(w), 0.0, dtype), "y")
    rows, _ = wq.wq_rms_norm_i8(x.cuda(), w.cuda(), eps=0.0)
    scales = rows.scales.cpu()
    assert (scales[[2, 5]] == 0).all() and scales[7].isnan() and (rows.codes[[2, 7]] == 0).all()
    assert np.array_equal(rows.codes.cpu().numpy()[ok], i8.quantize(f(x[ok]) * f(w))[0])
    real = ok + [2, 5]
    dx, dw = wq.wq_rms_norm_grad(dy[real].cuda(), x[real].cuda(), w.cuda(), ds[real].cuda(), eps=0.0)
    rx, bx, rw, bw = i8.norm_grad_bounds(f(dy[ok]), f(x[ok]), f(w), 0.0, f(ds[ok]), dtype)
    i8.assert_within(i8.to_host(dx)[:6], rx, bx, "dx")
    assert torch.equal(dx.cpu()[6:], ds[[2, 5]])
    i8.assert_within(i8.to_host(dw), rw, bw, "d_weight")


def test_gradients_of_very_long_rows(wq):
    """dx and d_weight of two rows of 2^28 + 72 ones of either sign: the lanes' and the waves' sums are whole numbers
    up to 2^24 and exact, so that 16 additions, inv and a few products are the errors."""
    import torch

    print("very long rows", flush=True)
    k = (1 << 28) + 72
    r, dy = ((torch.randint(0, 2, (2, k), device="cuda", dtype=torch.int8) * 2 - 1).to(torch.bfloat16) for _ in range(2))
    ds = torch.zeros_like(r)
    ds[:, -9:] = 4
    dx, dw = wq.wq_rms_norm_grad(dy, r, torch.ones(k, device="cuda", dtype=torch.bfloat16), ds)
    inv = 1 / np.sqrt(1 + 1e-6)
    mean = [float((dy[i] == r[i]).sum() * 2 - k) / k for i in range(2)]
    for at in (0, k // 3, k - 4000):
        s = slice(at, at + 4000)
        a, g, d = (t[:, s].double().cpu().numpy() for t in (r, dy, ds))
        ref = inv * (g - a * inv ** 2 * np.array(mean)[:, None]) + d
        i8.assert_within(i8.to_host(dx[:, s]), ref, np.abs(ref) * (i8.HALF["bf16"] + 26 * i8.U), "dx")
        ref = (g * a * inv).sum(0)
        i8.assert_within(i8.to_host(dw[s]), ref, 2 * 26 * i8.U, "d_weight")
