"""Quantisation to int8 and the products of two int8 operands on the GPU against the definitions in 64 bits
(i8_testutil): codes, scales and products bit for bit, SiLU(gate) * up within the bound derived there."""
import sys

import numpy as np
import pytest

import i8_testutil as i8
from i8_cases import DENSE, EXPERTS

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


def _cuda(a):
    import torch

    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _values(rng, n, k, dtype):
    import torch

    x = torch.from_numpy(rng.standard_normal((n, k)) * np.exp2(rng.integers(-20, 20, (n, 1)))).float()
    return x.to(torch.bfloat16) if dtype == "bf16" else x


# ---------------------------------------------------------------------------------------------
# quantisation
# ---------------------------------------------------------------------------------------------

# lengths: one element, shorter than a piece, every number of pieces a lane holds with and without a ragged
# end, rows of several waves, and rows that are read again (from 65537 bf16 or 32769 fp32 values on)
LENGTHS = [1, 3, 7, 8, 63, 64, 511, 512, 1027, 1111, 2048, 4096, 4160, 8200, 16384, 16391, 40000, 70003]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,k", [(5, k) for k in LENGTHS] + [(300, k) for k in (72, 520, 700, 1111, 3001, 8200, 12000)])
def test_quantize_rows(wq, dtype, n, k):
    _say("quantize", dtype, n, k)
    x = _values(np.random.default_rng(k), n, k, dtype)
    codes, a = i8.quantize(x.double().numpy())
    q = wq.wq_quantize_i8(x.cuda())
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    assert np.array_equal(q.scales.cpu().numpy(), i8.f32(a / 127))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(3, 64), (2, 5, 192), (1, 4160), (4, 3, 16384)])
def test_quantize_weights(wq, dtype, shape):
    _say("quantize weights", dtype, shape)
    x = _values(np.random.default_rng(2), int(np.prod(shape[:-1])), shape[-1], dtype)
    v = x.double().numpy()
    scale = i8.bf16(i8.f32(np.abs(v).max(1) / 127))
    codes = np.clip(np.round(v / scale[:, None]), -127, 127).astype(np.int8)
    w = wq.wq_quantize_i8_weight(x.reshape(shape).cuda())
    assert (w.format, w.group, w.experts, w.n, w.k) == (wq.FMT_INT8, 0, 1 if len(shape) == 2 else shape[0], *shape[-2:])
    assert np.array_equal(i8.to_host(w.scales).reshape(-1), scale)
    assert np.array_equal(w.codes.cpu().numpy().reshape(codes.shape), codes)
    back = i8.to_host(wq.wq_dequantize(w).view(__import__("torch").bfloat16)).reshape(codes.shape)
    assert np.array_equal(back, i8.bf16(codes * scale[:, None]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_edges(wq, dtype):
    """Half-way quotients, zeros of both signs, subnormal and the largest values, infinities and NaN."""
    import torch

    _say("quantize edges", dtype)
    big = float(torch.finfo(torch.bfloat16).max)
    rows = [[127, 63.5, -63.5, 0.5, -0.5, 1.5, 2.5, -2.5], [254, 1, 3, 5, 127, -253, 0, -0.0], [3, 1.5, -1.5, 0, 0, 0, 0, 0],
            [0.0, -0.0] * 4, [big, big / 2, -big, 1, 0, 0, 0, 0], [2.0 ** -133, 2.0 ** -132, -2.0 ** -131, 0, 0, 0, 0, 0],
            [1, 2, np.inf, 0, 0, 0, 0, 0], [1, 2, 3, 4, 5, 6, 7, -np.inf], [np.nan, 2, 3, 4, 5, 6, 7, 8],
            [0, 0, 0, 0, 0, 0, 0, np.nan], [0.1953125, 0.09765625, 0, 0, 0, 0, 0, 0]]
    x = torch.tensor(rows, dtype=torch.bfloat16).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    codes, a = i8.quantize(x.double().numpy())
    q = wq.wq_quantize_i8(x.cuda())
    assert np.array_equal(q.codes.cpu().numpy(), codes)
    assert np.array_equal(q.scales.cpu().numpy(), i8.f32(a / 127), equal_nan=True)
    w = wq.wq_quantize_i8_weight(torch.nn.functional.pad(x, (0, 56)).cuda())
    ok = np.isfinite(a)
    scale = i8.bf16(i8.f32(a / 127))
    assert np.array_equal(i8.to_host(w.scales)[0], scale, equal_nan=True)
    want = np.where((ok & (scale > 0))[:, None], x.double().numpy() / np.where(scale > 0, scale, 1)[:, None], 0)
    assert np.array_equal(w.codes.cpu().numpy()[0, :, :8], np.clip(np.round(np.where(ok[:, None], want, 0)), -127, 127))


def test_quantize_strided_and_empty(wq):
    import torch

    x = torch.randn(40, 128, device="cuda")[::3, :65]
    a, b = wq.wq_quantize_i8(x), wq.wq_quantize_i8(x.contiguous())
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    e = wq.wq_quantize_i8(torch.empty((0, 64), device="cuda"))
    assert e.codes.shape == (0, 64) and e.scales.shape == (0,)
    # the least k of the values: (1, 1)
    q = wq.wq_quantize_i8(torch.tensor([[-0.25]], device="cuda"))
    assert q.codes.item() == -127 and q.scales.item() == np.float32(0.25 / 127)


def test_quantize_many_rows(wq):
    """Rows in thousands of workgroups, each as the same row alone."""
    import torch

    x = torch.randn(100003, 72, device="cuda").to(torch.bfloat16)
    q = wq.wq_quantize_i8(x)
    f = x.double()
    a = f.abs().amax(1, keepdim=True)
    assert torch.equal(q.codes, torch.round(f * 127 / a).to(torch.int8))
    assert torch.equal(q.scales, (a[:, 0] / 127).float())


# ---------------------------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("case", DENSE, ids=lambda c: f"{c.kernel}-{c.m}x{c.n}x{c.k}")
def test_gemm(wq, case, out):
    import torch

    _say("gemm", case, out)
    rng = np.random.default_rng(case.m)
    c, s = i8.random_rows(rng, case.m, case.k)
    wc, ws = i8.random_weight(rng, 1, case.n, case.k)
    pad = torch.full((case.m * case.n + 64,), 7.0, device="cuda", dtype=torch.float32 if out == "f32" else torch.bfloat16)
    y = pad[: case.m * case.n].view(case.m, case.n)
    wq.wq_gemm_i8(i8.rows(wq, c, s), i8.weight(wq, wc, ws), y=y)
    assert np.array_equal(i8.to_host(y), i8.product_bits(c, s, wc[0], ws[0], out))
    assert (pad[case.m * case.n:] == 7).all()  # nothing behind the output


# streaming, few columns a workgroup, tiles of 64, 128, 128 x 256 and 256
@pytest.mark.parametrize("m,n,k", [(1, 16, 131008), (100, 1025, 65600), (32, 6145, 65600), (64, 3100, 131008), (70, 8190, 65600), (9, 8177, 65600),
                                   (200, 8190, 65600), (1300, 1701, 131008), (1440, 4100, 65600), (3100, 4097, 131008)])
def test_gemm_largest_sums(wq, m, n, k):
    """Every code -128, or 127 against -128: the largest sums of either sign stay in int32."""
    import torch

    _say("largest sums", m, n, k)
    for a, b in ((-128, -128), (127, -128), (127, 127)):
        x = wq.Int8Rows(torch.full((m, k), a, dtype=torch.int8, device="cuda"), torch.ones(m, device="cuda"))
        w = wq.PackedWeight(wq.FMT_INT8, n, k, 1, 0, codes=torch.full((1, n, k), b, dtype=torch.int8, device="cuda"),
                            scales=torch.ones((1, n), dtype=torch.bfloat16, device="cuda"))
        y = wq.wq_gemm_i8(x, w, dtype=torch.float32)
        assert (y == float(np.float32(a * b * k))).all()


def test_gemm_nan_rows_and_zero_scales(wq):
    """A row that was not finite gives NaN, a row of zeros zeros, and neither touches its neighbours."""
    import torch

    for m in (4, 300):
        x = torch.randn(m, 128, device="cuda").to(torch.bfloat16)
        x[1, 5], x[2] = float("inf"), 0
        w = wq.wq_quantize_i8_weight(torch.randn(600, 128, device="cuda"))
        y = wq.wq_gemm_i8(wq.wq_quantize_i8(x), w)
        assert y[1].isnan().all() and (y[2] == 0).all()
        rest = [i for i in range(m) if i != 1]
        assert y[rest].isfinite().all()


def _routing(rng, counts, t, topk):
    """(offsets, sorted pairs) with the given rows per expert; the other pairs are dropped."""
    flat = np.full(t * topk, -1, np.int32)
    flat[rng.permutation(t * topk)[: sum(counts)]] = np.repeat(np.arange(len(counts)), counts)
    order = [p for e in range(len(counts)) for p in np.nonzero(flat == e)[0]]
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32), np.array(order, np.int64), flat.reshape(t, topk)


@pytest.mark.parametrize("case", [c for c in EXPERTS if c.gate_up], ids=lambda c: f"{c.kernel}-{c.n}x{c.k}")
def test_gate_up(wq, case):
    import torch

    _say("gate_up", case)
    rng = np.random.default_rng(case.n)
    E = len(case.counts)
    offsets, order, ids = _routing(rng, case.counts, case.t, case.topk)
    off, pairs = wq.wq_moe_route(_cuda(ids), E)
    assert np.array_equal(off.cpu().numpy(), offsets)
    c, s = i8.random_rows(rng, case.t, case.k)
    s *= np.float32(2.0 ** -8)
    gate, up = i8.random_weight(rng, E, case.n, case.k), i8.random_weight(rng, E, case.n, case.k)
    p = case.t * case.topk
    h = torch.full((p, case.n), 7.0, dtype=torch.bfloat16, device="cuda")
    wq.wq_moe_gate_up_i8(i8.rows(wq, c, s), off, pairs, case.topk, i8.weight(wq, *gate), i8.weight(wq, *up), h=h)
    got = i8.to_host(h)
    for e in range(E):
        tok = order[offsets[e]: offsets[e + 1]] // case.topk
        ref, bound = i8.gate_up_bound(c[tok], s[tok], gate[0][e], gate[1][e], up[0][e], up[1][e])
        i8.assert_within(got[offsets[e]: offsets[e + 1]], ref, bound, f"expert {e}")
    assert (got[offsets[-1]:] == 7).all()  # rows of dropped pairs


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("case", [c for c in EXPERTS if not c.gate_up], ids=lambda c: f"{c.kernel}-{c.n}x{c.k}")
def test_down(wq, case, out):
    import torch

    _say("down", case, out)
    rng = np.random.default_rng(case.n)
    E, p = len(case.counts), case.t * case.topk
    offsets = np.concatenate([[0], np.cumsum(case.counts)]).astype(np.int32)
    c, s = i8.random_rows(rng, p, case.k)
    wc, ws = i8.random_weight(rng, E, case.n, case.k)
    d = torch.full((p, case.n), 7.0, dtype=torch.float32 if out == "f32" else torch.bfloat16, device="cuda")
    wq.wq_moe_down_i8(i8.rows(wq, c, s), _cuda(offsets), i8.weight(wq, wc, ws), d=d)
    got = i8.to_host(d)
    for e in range(E):
        a, b = offsets[e], offsets[e + 1]
        assert np.array_equal(got[a:b], i8.product_bits(c[a:b], s[a:b], wc[e], ws[e], out)), e
    assert (got[offsets[-1]:] == 7).all()


def test_no_rows_and_no_tokens(wq):
    import torch

    rng = np.random.default_rng(0)
    w = i8.weight(wq, *i8.random_weight(rng, 4, 64, 128))
    one = i8.weight(wq, *i8.random_weight(rng, 1, 64, 128))
    none = wq.wq_quantize_i8(torch.empty((0, 128), device="cuda"))
    assert wq.wq_gemm_i8(none, one).shape == (0, 64)
    off, pairs = wq.wq_moe_route(torch.empty((0, 2), dtype=torch.int32, device="cuda"), 4)
    assert wq.wq_moe_gate_up_i8(none, off, pairs, 2, w, w).shape == (0, 64)
    assert wq.wq_moe_down_i8(none, off, w).shape == (0, 64)
    # every pair dropped: nothing is written
    off, pairs = wq.wq_moe_route(torch.full((400, 2), -1, dtype=torch.int32, device="cuda"), 4)
    x = i8.rows(wq, *i8.random_rows(rng, 400, 128))
    h = torch.full((800, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    wq.wq_moe_gate_up_i8(x, off, pairs, 2, w, w, h=h)
    assert (h == 7).all()


def test_rows_beyond_32_bits(wq):
    """Codes and outputs that lie beyond 2^31 bytes: the last rows of 300000 x 8192, and outputs of 70000 x
    32000 fp32."""
    import torch

    _say("rows beyond 32 bits")
    n, k = 128, 8192
    w = i8.weight(wq, *i8.random_weight(np.random.default_rng(3), 1, n, k))
    codes = torch.randint(-128, 128, (300000, k), dtype=torch.int8, device="cuda")
    scales = torch.rand(300000, device="cuda") + 0.5
    y = wq.wq_gemm_i8(wq.Int8Rows(codes, scales), w)
    tail = wq.wq_gemm_i8(wq.Int8Rows(codes[-16:].clone(), scales[-16:].clone()), w)
    assert torch.equal(y[-16:], tail)
    del codes, y
    _say("outputs beyond 32 bits")
    c, s = i8.random_rows(np.random.default_rng(4), 70000, 64)
    wc, ws = i8.random_weight(np.random.default_rng(5), 1, 32000, 64)
    y = wq.wq_gemm_i8(i8.rows(wq, c, s), i8.weight(wq, wc, ws), dtype=torch.float32)
    assert np.array_equal(i8.to_host(y[-3:]), i8.product_bits(c[-3:], s[-3:], wc[0], ws[0], "f32"))
    assert np.array_equal(i8.to_host(y[:3]), i8.product_bits(c[:3], s[:3], wc[0], ws[0], "f32"))


def test_quantize_beyond_one_launch(wq):
    """More workgroups of 1024 threads than one launch holds."""
    import torch

    _say("beyond one launch")
    n, k = (1 << 22) + 5, 4104
    base = torch.randn((1024, k), device="cuda").to(torch.bfloat16)
    x = base.repeat(n // 1024 + 1, 1)[:n]
    q = wq.wq_quantize_i8(x)
    want = wq.wq_quantize_i8(base)
    for at in (0, n // 2, n - 5):
        rows = torch.arange(at, at + 5, device="cuda")
        assert torch.equal(q.codes[rows], want.codes[rows % 1024]) and torch.equal(q.scales[rows], want.scales[rows % 1024])
