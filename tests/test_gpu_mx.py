"""MXFP4 on the GPU against the definitions in 64 bits (mx_testutil): quantisation and decoding bit
for bit, the products within the bounds derived there, at sizes and in places where they can go
wrong."""
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


def _cuda(a, dtype=None):
    import torch

    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def _acts(rng, *shape):
    x = mx.bf16(rng.standard_normal(shape) * 1.0)
    x[..., :: 37] *= 16
    return x


# ---------------------------------------------------------------------------------------------
# quantisation and decoding
# ---------------------------------------------------------------------------------------------

def _edge_values():
    """Blocks of 32: every half-way point and its neighbours under scales from the least to the
    largest, zeros of both signs, subnormal and the largest values, infinities and NaN."""
    mid = np.array([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 5.5, 6], np.float32)
    rows = []
    for e in (-149, -140, -130, -127, -126, -125, -100, -1, 0, 1, 60, 122, 124):
        b = np.ldexp(np.concatenate([mid, -mid]).astype(np.float64), e).astype(np.float32)
        rows += [b, np.nextafter(b, np.float32(np.inf)), np.nextafter(b, np.float32(-np.inf)), b * np.float32(1.3)]
    big = np.zeros(32, np.float32)
    big[0] = np.finfo(np.float32).max
    rows += [np.zeros(32, np.float32), -np.zeros(32, np.float32), big]
    for bad in (np.inf, -np.inf, np.nan):
        r = rows[3].copy()
        r[31] = bad
        rows.append(r)
    if len(rows) % 2:
        rows.append(rows[0])
    return np.concatenate(rows).reshape(-1, 64)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_quantize_edges(wq, dtype):
    import torch

    _say("quantize edges", dtype)
    x = torch.from_numpy(_edge_values())
    if dtype == "bf16":
        x = x.to(torch.bfloat16)
    code, byte = mx.encode(x.double().numpy())
    q = wq.wq_quantize_mx(x.cuda())
    assert np.array_equal(q.qscale.cpu().numpy()[0], byte)
    assert np.array_equal(mx.unpack(q.codes.cpu().numpy()[0]), code)


@pytest.mark.parametrize("dtype,shape", [("f32", (1, 64)), ("bf16", (1, 64)), ("bf16", (17, 4160)), ("f32", (3, 5, 192)),
                                         ("bf16", (333, 64)), ("f32", (129, 1088))])
def test_quantize_and_dequantize(wq, dtype, shape):
    import torch

    _say("quantize", dtype, shape)
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal(shape) * np.exp2(rng.integers(-40, 40, (*shape[:-1], 1)))).float()
    if dtype == "bf16":
        x = x.to(torch.bfloat16)
    code, byte = mx.encode(x.double().numpy())
    q = wq.wq_quantize_mx(x.cuda())
    assert (q.experts, q.n, q.k) == (1 if len(shape) == 2 else shape[0], shape[-2], shape[-1])
    assert np.array_equal(q.qscale.cpu().numpy().reshape(byte.shape), byte)
    assert np.array_equal(mx.unpack(q.codes.cpu().numpy()).reshape(code.shape), code)
    back = mx.to_host(wq.wq_dequantize(q)).reshape(code.shape)
    assert np.array_equal(back, mx.values(code, byte))


def test_quantize_strided_and_empty(wq):
    import torch

    x = torch.randn(40, 128, device="cuda")[::3, :64]
    a, b = wq.wq_quantize_mx(x), wq.wq_quantize_mx(x.contiguous())
    assert torch.equal(a.codes, b.codes) and torch.equal(a.qscale, b.qscale)
    e = wq.wq_quantize_mx(torch.empty((0, 64), device="cuda"))
    assert e.n == 0 and e.codes.numel() == 0


def test_dequantize_every_code_and_scale(wq):
    code = np.tile(np.arange(32, dtype=np.uint8) % 16, (256, 2))
    byte = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 2, 1)
    ref = mx.values(code, byte)
    got = mx.to_host(wq.wq_dequantize(mx.weight(wq, code[None], byte[None])))[0]
    fits = np.abs(ref) < 2.0 ** 128
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    assert np.array_equal(got[fits], ref[fits])
    assert np.array_equal(np.signbit(got[fits]), np.signbit(ref[fits]))
    over = ~fits & ~np.isnan(ref)
    assert np.array_equal(got[over], np.sign(ref[over]) * np.inf)


# ---------------------------------------------------------------------------------------------
# dense products
# ---------------------------------------------------------------------------------------------

# decode, single-staging and tiled kernels; n, k ragged in every way the format allows
BF16_SIZES = [(1, 16, 64), (1, 1111, 512), (5, 40, 1024), (16, 77, 4096), (17, 130, 192), (24, 96, 4160), (32, 257, 320),
              (33, 100, 64), (64, 65, 448), (300, 530, 704), (129, 256, 256)]


@pytest.mark.parametrize("m,n,k", BF16_SIZES)
def test_gemm_bf16_activations(wq, m, n, k):
    import torch

    _say("gemm bf16", m, n, k)
    rng = np.random.default_rng(m * n + k)
    code, byte = mx.random_codes(rng, 1, n, k)
    x = _acts(rng, m, k)
    ref, mag = mx.product(x, mx.values(code, byte)[0])
    y = wq.wq_gemm(_cuda(x, torch.bfloat16), mx.weight(wq, code, byte))
    mx.assert_within(mx.to_host(y), ref, mx.sum_bound(ref, mag, k, "bf16"), f"gemm {m} {n} {k}")


MX_SIZES = [(1, 1, 64), (1, 16, 64), (1, 1111, 512), (2, 64, 4160), (16, 77, 4096), (17, 130, 192), (32, 257, 320),
            (33, 100, 64), (64, 65, 448), (65, 4096, 128), (100, 33, 8192), (128, 128, 256), (129, 255, 576),
            (300, 530, 704), (256, 512, 1024), (513, 300, 1088)]


@pytest.mark.parametrize("m,n,k", MX_SIZES)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_gemm_mx(wq, m, n, k, out):
    import torch

    _say("gemm_mx", m, n, k, out)
    rng = np.random.default_rng(m + n * k)
    code, byte = mx.random_codes(rng, 1, n, k)
    xc, xb = mx.encode(_acts(rng, m, k))
    ref, mag = mx.product(mx.values(xc, xb), mx.values(code, byte)[0])
    y = wq.wq_gemm_mx(mx.weight(wq, xc[None], xb[None]), mx.weight(wq, code, byte),
                      dtype=torch.float32 if out == "f32" else None)
    assert y.dtype == (torch.float32 if out == "f32" else torch.bfloat16)
    mx.assert_within(mx.to_host(y), ref, mx.sum_bound(ref, mag, k, out), f"gemm_mx {m} {n} {k} {out}")


@pytest.mark.parametrize("m", [1, 16, 40, 150, 300])
@pytest.mark.parametrize("k", [64, 192, 576])
def test_nan_blocks_stay_in_their_row(wq, m, k):
    """A NaN block makes its row (of x) or column (of W) NaN and no other value: also where a
    kernel's step runs past the row's end, into the next row's first block."""
    import torch

    _say("nan blocks", m, k)
    rng = np.random.default_rng(5)
    n = 50
    code, byte = mx.random_codes(rng, 1, n, k)
    byte[0, 7, 0] = byte[0, 20, -1] = 255
    w = mx.weight(wq, code, byte)
    xv = _acts(rng, m, k)
    ref, mag = mx.product(xv, mx.values(code, byte)[0])
    assert np.isnan(ref).sum() == 2 * m
    bound = mx.sum_bound(np.nan_to_num(ref), np.nan_to_num(mag), k, "bf16")
    mx.assert_within(mx.to_host(wq.wq_gemm(_cuda(xv, torch.bfloat16), w)), ref, bound, "bf16 activations")
    xc, xb = mx.encode(xv)
    xb[m // 2, 0] = 255
    xb[m - 1, -1] = 255
    ref, mag = mx.product(mx.values(xc, xb), mx.values(code, byte)[0])
    bound = mx.sum_bound(np.nan_to_num(ref), np.nan_to_num(mag), k, "bf16")
    mx.assert_within(mx.to_host(wq.wq_gemm_mx(mx.weight(wq, xc[None], xb[None]), w)), ref, bound, "mx activations")


@pytest.mark.parametrize("m", [3, 24, 64, 200])
def test_products_at_extreme_scales(wq, m):
    """Weights near the largest and the least bf16 values, activations the other way round."""
    import torch

    rng = np.random.default_rng(9)
    n, k = 48, 256
    for shift in (110, -118):
        _say("extreme scales", m, shift)
        code, byte = mx.random_codes(rng, 1, n, k)
        byte = (byte.astype(int) + shift).clip(0, 250).astype(np.uint8)
        w = mx.weight(wq, code, byte)
        x = np.ldexp(_acts(rng, m, k), -shift)
        ref, mag = mx.product(x, mx.values(code, byte)[0])
        got = mx.to_host(wq.wq_gemm(_cuda(x, torch.bfloat16), w))
        mx.assert_within(got, ref, mx.sum_bound(ref, mag, k, "bf16"), "bf16")
        xc, xb = mx.encode(x)
        ref, mag = mx.product(mx.values(xc, xb), mx.values(code, byte)[0])
        got = mx.to_host(wq.wq_gemm_mx(mx.weight(wq, xc[None], xb[None]), w))
        mx.assert_within(got, ref, mx.sum_bound(ref, mag, k, "bf16"), "mx")


def test_gemm_mx_empty_and_refusals(wq):
    import torch

    rng = np.random.default_rng(2)
    w = mx.weight(wq, *mx.random_codes(rng, 1, 32, 128))
    x = wq.wq_quantize_mx(torch.randn(4, 128, device="cuda"))
    assert wq.wq_gemm_mx(wq.wq_quantize_mx(torch.empty((0, 128), device="cuda")), w).shape == (0, 32)
    with pytest.raises(ValueError, match="k = 64"):
        wq.wq_gemm_mx(wq.wq_quantize_mx(torch.randn(4, 64, device="cuda")), w)
    with pytest.raises(ValueError, match="one MXFP4 matrix"):
        wq.wq_gemm_mx(wq.wq_quantize_mx(torch.randn(2, 4, 128, device="cuda")), w)
    with pytest.raises(ValueError, match="shape"):
        wq.wq_gemm_mx(x, w, y=torch.empty((4, 31), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError, match="neither"):
        wq.wq_gemm_mx(x, w, y=torch.empty((4, 32), dtype=torch.float16, device="cuda"))
    with pytest.raises(TypeError, match="PackedWeight"):
        wq.wq_gemm_mx(torch.randn(4, 128, device="cuda").bfloat16(), w)
    with pytest.raises(ValueError, match="codes"):
        wq.wq_gemm_mx(wq.PackedWeight(wq.FMT_MXFP4, 5, 128, 1, 32, codes=x.codes, qscale=x.qscale), w)
    with pytest.raises(ValueError, match="WQ_ERR_UNSUPPORTED"):
        wq.wq_gemm_mx(x, wq.wq_quantize_ccq(torch.randn(32, 128, device="cuda")))


# ---------------------------------------------------------------------------------------------
# experts
# ---------------------------------------------------------------------------------------------

def _ids(rng, t, topk, E, kind):
    if kind == "one":  # every pair on one expert, the others empty
        return np.full((t, topk), E // 2, np.int32)
    ids = rng.integers(0, E, (t, topk)).astype(np.int32)
    if kind == "skewed":
        ids[rng.random((t, topk)) < 0.7] = 1
        ids[ids == 0] = 1  # expert 0 empty
    if kind == "dropped":
        ids[rng.random((t, topk)) < 0.3] = E
        ids[0] = -1  # a token without any expert
    return ids


# (t, topk, E, inter, hidden, routing): from one token to many rows per expert
MOE = [(1, 1, 4, 32, 64, "any"), (3, 2, 8, 100, 192, "any"), (16, 8, 8, 65, 512, "any"), (40, 4, 4, 130, 320, "dropped"),
       (70, 3, 5, 96, 256, "skewed"), (300, 2, 3, 260, 448, "skewed"), (257, 1, 2, 64, 1088, "one"),
       (700, 2, 4, 129, 128, "dropped"), (24, 6, 64, 48, 128, "any")]


@pytest.mark.parametrize("t,topk,E,inter,hidden,kind", MOE)
def test_moe_products_mx(wq, t, topk, E, inter, hidden, kind):
    import torch

    _say("moe mx", t, topk, E, inter, hidden, kind)
    rng = np.random.default_rng(t + hidden)
    ids = _ids(rng, t, topk, E, kind)
    off, order, _ = mx.route(ids, E)
    offsets, pairs = wq.wq_moe_route(_cuda(ids), E)
    assert np.array_equal(offsets.cpu().numpy(), off)
    xc, xb = mx.encode(_acts(rng, t, hidden))
    x = mx.values(xc, xb)
    g, u = (mx.random_codes(rng, E, inter, hidden) for _ in range(2))
    P, live = t * topk, len(order)
    h = torch.full((P, inter), 7.0, dtype=torch.bfloat16, device="cuda")
    got = mx.to_host(wq.wq_moe_gate_up_mx(mx.weight(wq, xc[None], xb[None]), offsets, pairs, topk,
                                          mx.weight(wq, *g), mx.weight(wq, *u), h=h))
    assert np.all(got[live:] == 7.0), "rows behind the last expert's were written"
    gv, uv = mx.values(*g), mx.values(*u)
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        xe = x[order[rows] // topk]
        (a, am), (b, bm) = mx.product(xe, gv[e]), mx.product(xe, uv[e])
        ref, bound = mx.gate_up_bound(a, am, b, bm, hidden)
        mx.assert_within(got[rows], ref, bound, f"gate_up expert {e}")
    # down on rows of its own
    n, k = hidden, 64 * ((inter + 63) // 64)
    hc, hb = mx.encode(_acts(rng, P, k))
    d = mx.random_codes(rng, E, n, k)
    dv, hv = mx.values(*d), mx.values(hc, hb)
    for out, dt in (("bf16", torch.bfloat16), ("f32", torch.float32)):
        o = torch.full((P, n), 7.0, dtype=dt, device="cuda")
        got = mx.to_host(wq.wq_moe_down_mx(mx.weight(wq, hc[None], hb[None]), offsets, mx.weight(wq, *d), d=o))
        assert np.all(got[live:] == 7.0)
        for e in range(E):
            rows = slice(off[e], off[e + 1])
            ref, mag = mx.product(hv[rows], dv[e])
            mx.assert_within(got[rows], ref, mx.sum_bound(ref, mag, k, out), f"down expert {e} {out}")


@pytest.mark.parametrize("t,topk,E,inter,hidden", [(1, 2, 4, 64, 256), (12, 4, 8, 128, 512), (64, 4, 8, 192, 320),
                                                  (400, 2, 4, 256, 448)])
def test_moe_bf16_activations(wq, t, topk, E, inter, hidden):
    """The stages of the bf16-activation FFN on MXFP4 experts, and the FFN as their sequence."""
    import torch

    _say("moe bf16", t, topk, E, inter, hidden)
    rng = np.random.default_rng(t)
    ids = _ids(rng, t, topk, E, "any")
    wts = rng.random((t, topk)).astype(np.float32)
    off, order, _ = mx.route(ids, E)
    offsets, pairs = wq.wq_moe_route(_cuda(ids), E)
    x = _acts(rng, t, hidden)
    g, u, d = (mx.random_codes(rng, E, *s) for s in ((inter, hidden), (inter, hidden), (hidden, inter)))
    xd, gd, ud, dd = _cuda(x, torch.bfloat16), *(mx.weight(wq, *w) for w in (g, u, d))
    h = wq.wq_moe_gate_up(xd, offsets, pairs, topk, gd, ud)
    hv = mx.to_host(h)
    out = wq.wq_moe_down(h, t, topk, offsets, pairs, dd)
    ov = mx.to_host(out)
    gv, uv, dv = mx.values(*g), mx.values(*u), mx.values(*d)
    for e in range(E):
        r = order[off[e]:off[e + 1]]
        (a, am), (b, bm) = mx.product(x[r // topk], gv[e]), mx.product(x[r // topk], uv[e])
        ref, bound = mx.gate_up_bound(a, am, b, bm, hidden)
        mx.assert_within(hv[off[e]:off[e + 1]], ref, bound, f"gate_up {e}")
        ref, mag = mx.product(hv[off[e]:off[e + 1]], dv[e])
        mx.assert_within(ov[r], ref, mx.sum_bound(ref, mag, inter, "f32"), f"down {e}")
    y = wq.wq_moe_combine(out, _cuda(wts))
    assert torch.equal(y, wq.wq_moe_ffn(xd, _cuda(ids), _cuda(wts), gd, ud, dd))


# ---------------------------------------------------------------------------------------------
# runs, streams, graphs
# ---------------------------------------------------------------------------------------------

def _ffn(wq, x, ids, wts, gate, up, down, E, topk):
    """The MXFP4 FFN as a user writes it."""
    offsets, pairs = wq.wq_moe_route(ids, E)
    positions = wq.wq_moe_positions(ids, offsets, pairs)
    h = wq.wq_moe_gate_up_mx(wq.wq_quantize_mx(x), offsets, pairs, topk, gate, up)
    d = wq.wq_moe_down_mx(wq.wq_quantize_mx(h), offsets, down)
    return wq.wq_moe_unpermute(d, positions, wts), h, d


@pytest.mark.parametrize("t", [1, 20, 300])
def test_mx_ffn_run(wq, t):
    """quantise -> gate+up -> quantise -> down -> back, each step against 64 bits from the step
    before it."""
    import torch

    _say("mx ffn", t)
    E, topk, H, I = 8, 2, 320, 192
    rng = np.random.default_rng(t)
    ids = _ids(rng, t, topk, E, "any")
    wts = rng.random((t, topk)).astype(np.float32)
    off, order, pos = mx.route(ids, E)
    x = _acts(rng, t, H)
    mats = [mx.random_codes(rng, E, *s) for s in ((I, H), (I, H), (H, I))]
    y, h, d = _ffn(wq, _cuda(x, torch.bfloat16), _cuda(ids), _cuda(wts), *(mx.weight(wq, *w) for w in mats), E, topk)
    y, h, d = mx.to_host(y), mx.to_host(h), mx.to_host(d)
    gv, uv, dv = (mx.values(*w) for w in mats)
    xq, hq = mx.values(*mx.encode(x)), mx.values(*mx.encode(h))
    for e in range(E):
        r = order[off[e]:off[e + 1]] // topk
        (a, am), (b, bm) = mx.product(xq[r], gv[e]), mx.product(xq[r], uv[e])
        mx.assert_within(h[off[e]:off[e + 1]], *mx.gate_up_bound(a, am, b, bm, H), "h")
        ref, mag = mx.product(hq[off[e]:off[e + 1]], dv[e])
        mx.assert_within(d[off[e]:off[e + 1]], ref, mx.sum_bound(ref, mag, I, "bf16"), "d")
    w64 = wts.astype(np.float64)[:, :, None]
    ref, mag = (w64 * d[pos]).sum(1), (w64 * np.abs(d[pos])).sum(1)
    mx.assert_within(y, ref, mx.sum_bound(ref, mag, 2 * topk, "bf16"), "y")


@pytest.mark.parametrize("m,n,k", [(1, 300, 512), (40, 256, 320), (520, 512, 576)])
def test_products_repeat_bit_for_bit(wq, m, n, k):
    import torch

    rng = np.random.default_rng(3)
    w = mx.weight(wq, *mx.random_codes(rng, 1, n, k))
    x = torch.randn(m, k, device="cuda").bfloat16()
    q = wq.wq_quantize_mx(x)
    a, b = wq.wq_gemm_mx(q, w), wq.wq_gemm(x, w)
    for _ in range(5):
        assert torch.equal(a, wq.wq_gemm_mx(q, w)) and torch.equal(b, wq.wq_gemm(x, w))


def test_two_streams_at_once(wq):
    import torch

    rng = np.random.default_rng(4)
    w = mx.weight(wq, *mx.random_codes(rng, 1, 512, 1024))
    xs = [torch.randn(m, 1024, device="cuda").bfloat16() for m in (3, 400)]
    refs = [wq.wq_gemm_mx(wq.wq_quantize_mx(x), w) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    outs = [[], []]
    for _ in range(8):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(wq.wq_gemm_mx(wq.wq_quantize_mx(xs[i]), w))
    torch.cuda.synchronize()
    for i in range(2):
        for o in outs[i]:
            assert torch.equal(o, refs[i])


@pytest.mark.parametrize("t", [4, 600])
def test_mx_ffn_captured(wq, t):
    import torch

    _say("mx ffn graph", t)
    E, topk, H, I = 4, 2, 256, 128
    rng = np.random.default_rng(t)
    mats = [mx.weight(wq, *mx.random_codes(rng, E, *s)) for s in ((I, H), (I, H), (H, I))]
    new = lambda: (torch.randn(t, H, device="cuda").bfloat16(), _cuda(_ids(rng, t, topk, E, "dropped")),
                   torch.rand(t, topk, device="cuda"))
    live = new()
    run = lambda a: _ffn(wq, *a, *mats, E, topk)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(live)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = run(live)
    for _ in range(4):
        other = new()
        want = run(other)
        for a, b in zip(live, other):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


# ---------------------------------------------------------------------------------------------
# sizes that reach every kernel of the products: the references multiply in float64 on the GPU
# ---------------------------------------------------------------------------------------------

def _mm64(x, w):
    """(x w^T, magnitudes) in fp64 of host values, multiplied on the GPU."""
    import torch

    a, b = torch.from_numpy(x).cuda(), torch.from_numpy(np.ascontiguousarray(w.T)).cuda()
    return torch.mm(a, b).cpu().numpy(), torch.mm(a.abs(), b.abs()).cpu().numpy()


# dense tiles of 64 x 64, 128 x 128, 128 x 256 (two buffers, one buffer), 256 x 256; k with a stage that
# ends inside, n that no 16-byte piece divides
BIG = [(513, 900, 1088), (1300, 1700, 448), (1500, 4100, 320), (4100, 4099, 256), (4111, 4096, 576), (3100, 4097, 2112)]


@pytest.mark.parametrize("m,n,k", BIG)
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_gemm_mx_every_tile(wq, m, n, k, out):
    import torch

    _say("gemm_mx big", m, n, k, out)
    rng = np.random.default_rng(m)
    code, byte = mx.encode(rng.standard_normal((n, k)) * np.exp2(rng.integers(-2, 3, (n, 1))))
    xc, xb = mx.encode(mx.bf16(rng.standard_normal((m, k))))
    y = torch.full((m + 1, n), 9.0, dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")
    wq.wq_gemm_mx(mx.weight(wq, xc[None], xb[None]), mx.weight(wq, code[None], byte[None]), y=y[:m])
    assert bool((y[m] == 9.0).all()), "the row behind the last one was written"
    ref, mag = _mm64(mx.values(xc, xb), mx.values(code, byte))
    mx.assert_within(mx.to_host(y[:m]), ref, mx.sum_bound(ref, mag, k, out), f"{m} {n} {k}")


@pytest.mark.parametrize("m,n,k", [(40, 28801, 192), (100, 17001, 64), (1400, 2000, 320), (2000, 1537, 448)])
def test_gemm_bf16_activations_tiled(wq, m, n, k):
    import torch

    _say("gemm bf16 tiled", m, n, k)
    rng = np.random.default_rng(m)
    code, byte = mx.encode(rng.standard_normal((n, k)))
    byte[n // 2, -1] = 255
    x = mx.bf16(rng.standard_normal((m, k)))
    y = wq.wq_gemm(_cuda(x, torch.bfloat16), mx.weight(wq, code[None], byte[None]))
    ref, mag = _mm64(x, mx.values(code, byte))
    mx.assert_within(mx.to_host(y), ref, mx.sum_bound(np.nan_to_num(ref), np.nan_to_num(mag), k, "bf16"), "tiled")


# (t, topk, E, n, k, routing) of gate+up and of down: 128 x 256 tiles with two buffers, 128 x 128, 128 x 256
# with one buffer, 256 x 256 with small tiles beside, more experts than a wave's lanes, none with a row
MOE_BIG = [(40, 4, 8, 2100, 320, "any"), (200, 2, 4, 300, 320, "dropped"), (300, 2, 3, 2500, 448, "skewed"),
           (700, 2, 2, 9500, 2112, "skewed"), (300, 4, 130, 700, 256, "any"), (60, 2, 4, 4000, 256, "none")]


@pytest.mark.parametrize("t,topk,E,n,k,kind", MOE_BIG)
def test_moe_mx_every_tile(wq, t, topk, E, n, k, kind):
    import torch

    _say("moe mx big", t, topk, E, n, k, kind)
    rng = np.random.default_rng(t + n)
    ids = np.full((t, topk), E, np.int32) if kind == "none" else _ids(rng, t, topk, E, kind)
    off, order, _ = mx.route(ids, E)
    offsets, pairs = wq.wq_moe_route(_cuda(ids), E)
    g, u = (mx.encode(rng.standard_normal((E, n, k))) for _ in range(2))
    P, live = t * topk, len(order)
    gd, ud = mx.weight(wq, *g), mx.weight(wq, *u)
    for rows, gate_up in ((t, True), (P, False)):
        xc, xb = mx.encode(mx.bf16(rng.standard_normal((rows, k)) / k ** 0.5))
        x, xd = mx.values(xc, xb), mx.weight(wq, xc[None], xb[None])
        o = torch.full((P, n), 7.0, dtype=torch.bfloat16, device="cuda")
        if gate_up:
            wq.wq_moe_gate_up_mx(xd, offsets, pairs, topk, gd, ud, h=o)
        else:
            wq.wq_moe_down_mx(xd, offsets, gd, d=o)
        got = mx.to_host(o)
        assert np.all(got[live:] == 7.0), "rows behind the last expert's were written"
        for e in range(E):
            r = slice(off[e], off[e + 1])
            if off[e] == off[e + 1]:
                continue
            xe = x[order[r] // topk] if gate_up else x[r]
            a, am = _mm64(xe, mx.values(g[0][e], g[1][e]))
            if gate_up:
                b, bm = _mm64(xe, mx.values(u[0][e], u[1][e]))
                ref, bound = mx.gate_up_bound(a, am, b, bm, k)
            else:
                ref, bound = a, mx.sum_bound(a, am, k, "bf16")
            mx.assert_within(got[r], ref, bound, f"expert {e} gate_up {gate_up}")
