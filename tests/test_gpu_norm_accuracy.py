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
