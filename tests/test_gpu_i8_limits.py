"""The int8 products at their limits on the GPU: few rows by many columns, hundreds of experts, codes beyond 2^31 bytes
and the largest dense weight."""
import numpy as np
import pytest

import i8_testutil as i8
from i8_many_experts import MANY, counts_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wq():
    import torch

    import weight_only_bit_amd as wq

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    wq.lib()
    return wq


def _cuda(a):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("m", [33, 48, 64])
def test_few_rows_by_many_columns(wq, m, out):
    import torch

    print("few rows", m, out, flush=True)
    rng = np.random.default_rng(m)
    n, k = 49157, 192
    c, s = i8.random_rows(rng, m, k)
    wc, ws = i8.random_weight(rng, 1, n, k)
    y = wq.wq_gemm_i8(i8.rows(wq, c, s), i8.weight(wq, wc, ws), dtype=torch.float32 if out == "f32" else torch.bfloat16)
    assert np.array_equal(i8.to_host(y), i8.product_bits(c, s, wc[0], ws[0], out))


@pytest.mark.parametrize("case", MANY, ids=lambda c: f"{c.kernel}-{'up' if c.gate_up else 'down'}-{c.experts}")
def test_many_experts(wq, case):
    import torch

    print("many experts", case, flush=True)
    rng = np.random.default_rng(case.k + case.n)
    E, pairs, counts = case.experts, case.t * case.topk, counts_of(case)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    wc, ws = i8.random_weight(rng, E, case.n, case.k)
    out = torch.full((pairs, case.n), 7.0, dtype=torch.bfloat16, device="cuda")
    if case.gate_up:
        flat = np.full(pairs, -1, np.int32)
        flat[rng.permutation(pairs)[: offsets[-1]]] = np.repeat(np.arange(E), counts)
        off, order = wq.wq_moe_route(_cuda(flat.reshape(case.t, case.topk)), E)
        assert np.array_equal(off.cpu().numpy(), offsets)
        c, s = i8.random_rows(rng, case.t, case.k)
        s *= np.float32(2.0 ** -8)
        uc, us = i8.random_weight(rng, E, case.n, case.k)
        wq.wq_moe_gate_up_i8(i8.rows(wq, c, s), off, order, case.topk, i8.weight(wq, wc, ws), i8.weight(wq, uc, us), h=out)
    else:
        c, s = i8.random_rows(rng, pairs, case.k)
        wq.wq_moe_down_i8(i8.rows(wq, c, s), _cuda(offsets), i8.weight(wq, wc, ws), d=out)
    got = i8.to_host(out)
    for e in range(E):
        at = slice(offsets[e], offsets[e + 1])
        if case.gate_up:
            tok = np.nonzero(flat == e)[0] // case.topk
            if len(tok):
                i8.assert_within(got[at], *i8.gate_up_bound(c[tok], s[tok], wc[e], ws[e], uc[e], us[e]), f"expert {e}")
        else:
            assert np.array_equal(got[at], i8.product_bits(c[at], s[at], wc[e], ws[e], "bf16")), e
    assert (got[offsets[-1]:] == 7).all()


# streaming, tiles of 128 x 256 and of 256 x 256, by the rows that 40 experts have
@pytest.mark.parametrize("pairs", [40, 640, 5200])
def test_codes_beyond_32_bits(wq, pairs):
    """40 experts of 64 MiB: the last ones' codes lie beyond 2^31 bytes; their rows are what each alone gives."""
    import torch

    print("codes beyond 32 bits", pairs, flush=True)
    E, n, k = 40, 8192, 8192
    g = torch.Generator(device="cuda").manual_seed(pairs)
    some = lambda *s: torch.randint(-128, 128, s, dtype=torch.int8, device="cuda", generator=g)
    scales = lambda *s: (torch.rand(s, device="cuda", generator=g) * 1e-3).to(torch.bfloat16)
    gate, up = (wq.PackedWeight(wq.FMT_INT8, n, k, E, 0, codes=some(E, n, k), scales=scales(E, n)) for _ in range(2))
    one = lambda w, e: wq.PackedWeight(wq.FMT_INT8, n, k, 1, 0, codes=w.codes[e: e + 1].clone(), scales=w.scales[e: e + 1].clone())
    ids = torch.randint(0, E, (pairs, 1), device="cuda", dtype=torch.int32, generator=g)
    ids[:3] = E - 1
    off, order = wq.wq_moe_route(ids, E)
    x = wq.Int8Rows(some(pairs, k), torch.rand(pairs, device="cuda", generator=g) * 1e-4)
    h = wq.wq_moe_gate_up_i8(x, off, order, 1, gate, up)
    d = wq.wq_moe_down_i8(x, off, gate, dtype=torch.float32)
    at = off.tolist()
    for e in (0, E // 2, E - 2, E - 1):
        a, b = at[e], at[e + 1]
        if a == b:
            continue
        alone = wq.Int8Rows(x.codes[a:b].clone(), x.scales[a:b].clone())
        assert torch.equal(d[a:b], wq.wq_gemm_i8(alone, one(gate, e), dtype=torch.float32)), e
        rows = order[a:b].long()
        alone = wq.Int8Rows(x.codes[rows], x.scales[rows])
        ends = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        mine = torch.arange(b - a, dtype=torch.int32, device="cuda")
        assert torch.equal(h[a:b], wq.wq_moe_gate_up_i8(alone, ends, mine, 1, one(gate, e), one(up, e))), e


@pytest.mark.parametrize("m", [20, 64])
@pytest.mark.parametrize("n", [33554416, 33554431])
def test_largest_dense_weight(wq, m, n):
    """Codes of 2^31 - 1024 bytes, the tiles' last size, and of 2^31 - 64, which streams."""
    import torch

    print("largest weight", m, n, flush=True)
    k = 64
    codes = torch.randint(-128, 128, (1, n, k), dtype=torch.int8, device="cuda")
    scales = torch.rand((1, n), device="cuda").to(torch.bfloat16)
    x = wq.Int8Rows(torch.randint(-128, 128, (m, k), dtype=torch.int8, device="cuda"), torch.rand(m, device="cuda"))
    y = wq.wq_gemm_i8(x, wq.PackedWeight(wq.FMT_INT8, n, k, 1, 0, codes=codes, scales=scales))
    for a in (0, n // 2, n - 1000):
        w = wq.PackedWeight(wq.FMT_INT8, 1000, k, 1, 0, codes=codes[:, a: a + 1000].clone(), scales=scales[:, a: a + 1000].clone())
        assert torch.equal(y[:, a: a + 1000], wq.wq_gemm_i8(x, w)), a


def test_strided_inputs_are_refused(wq):
    """Rows that are not contiguous: only the quantisers copy them."""
    import torch

    wide = torch.randn((6, 256), device="cuda")
    x, w = wide[:, :128], torch.ones(128, device="cuda")
    c = x.contiguous()
    rows = wq.wq_quantize_i8(c)
    weight = wq.wq_quantize_i8_weight(torch.randn((64, 128), device="cuda"))
    ids = torch.zeros((6, 4), dtype=torch.int32, device="cuda")
    off, pairs = wq.wq_moe_route(ids[:, :2].contiguous(), 1)
    codes = torch.zeros((6, 256), dtype=torch.int8, device="cuda")[:, :128]
    strided = wq.Int8Rows(codes, rows.scales)
    counts = torch.ones(129, dtype=torch.int32, device="cuda")
    for call in (lambda: wq.wq_rms_norm(x, w), lambda: wq.wq_rms_norm(c, w, x), lambda: wq.wq_rms_norm(c, w, y=x),
                 lambda: wq.wq_rms_norm_i8(x, w), lambda: wq.wq_rms_norm_i8(c, w, rows=strided),
                 lambda: wq.wq_rms_norm_grad(x, c, w), lambda: wq.wq_rms_norm_grad(c, x, w),
                 lambda: wq.wq_rms_norm_grad(c, c, w, x), lambda: wq.wq_rms_norm_grad(c, c, w, dx=x),
                 lambda: wq.wq_gemm_i8(strided, weight), lambda: wq.wq_gemm_i8(rows, weight, y=wide[:, :64]),
                 lambda: wq.wq_moe_gate_up_i8(strided, off, pairs, 2, weight, weight), lambda: wq.wq_moe_down_i8(strided, off, weight),
                 lambda: wq.wq_moe_balance_loss(x, ids), lambda: wq.wq_moe_balance_loss(c, ids[:, :2]),
                 lambda: wq.wq_moe_balance_loss_grad(x, ids, counts), lambda: wq.wq_moe_balance_loss_grad(c, ids, counts, d_logits=x)):
        with pytest.raises(ValueError, match="contiguous"):
            call()
    assert torch.equal(wq.wq_quantize_i8(x).codes, rows.codes)
