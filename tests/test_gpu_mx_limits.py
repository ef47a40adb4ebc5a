"""The products of two MXFP4 operands where sizes leave 32 bits or one launch: more rows than a grid's z
extent holds, more threads than 2^32, arrays longer than 4 GiB, the most experts, none of anything.  Values
are checked in float64 where the limits lie."""
import numpy as np
import pytest

import mx_testutil as mx

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wq():
    import torch

    import weight_only_bit_amd as wq

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    wq.lib()
    yield wq
    torch.cuda.empty_cache()


@pytest.fixture(autouse=True)
def _room():
    import torch

    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB of free device memory")


def _random(wq, E, n, k, seed):
    """Uniform codes (two per byte, as stored) under scales over seven octaves."""
    import torch

    g = torch.Generator(device="cuda").manual_seed(seed)
    return wq.PackedWeight(
        wq.FMT_MXFP4, n, k, E, 32, codes=torch.randint(0, 256, (E, n, k // 2), generator=g, device="cuda", dtype=torch.uint8),
        qscale=torch.randint(120, 127, (E, n, k // 32), generator=g, device="cuda", dtype=torch.uint8))


def _values(w, rows, e=0):
    """fp64 values of some rows, on the host."""
    return mx.values(mx.unpack(w.codes[e, rows].cpu().numpy()), w.qscale[e, rows].cpu().numpy())


def _check(got, x, w, k, out, what):
    ref, mag = mx.product(x, w)
    mx.assert_within(mx.to_host(got), ref, mx.sum_bound(ref, mag, k, out), what)


@pytest.mark.parametrize("n", [1, 3])
def test_rows_beyond_one_launch(wq, n):
    import torch

    m, k = 65535 * 32 + 37, 64
    print("rows", m, n, k, flush=True)
    x, w = _random(wq, 1, m, k, 1), _random(wq, 1, n, k, 2)
    wv = _values(w, slice(None))
    y = wq.wq_gemm_mx(x, w)
    xb = wq.wq_dequantize(x)[0].view(torch.bfloat16)
    yb = wq.wq_gemm(xb, w)
    for rows in (slice(0, 300), slice(65535 * 16 - 50, 65535 * 16 + 50), slice(65535 * 32 - 100, m)):
        _check(y[rows], _values(x, rows), wv, k, "bf16", f"rows {rows}")
        _check(yb[rows], mx.to_host(xb[rows]), wv, k, "bf16", f"bf16 activations, rows {rows}")


def test_more_threads_than_32_bits(wq):
    m, n, k = (1 << 17) + 33, (1 << 16) + 7, 64  # 256 threads for 32 x 16 outputs
    print("threads", m, n, k, flush=True)
    x, w = _random(wq, 1, m, k, 3), _random(wq, 1, n, k, 4)
    y = wq.wq_gemm_mx(x, w)
    for rows in (slice(0, 40), slice(m // 2, m // 2 + 40), slice(m - 40, m)):
        for cols in (slice(0, 70), slice(n // 2, n // 2 + 70), slice(n - 70, n)):
            _check(y[rows, cols], _values(x, rows), _values(w, cols), k, "bf16", f"{rows} {cols}")


def test_activations_beyond_4_gib(wq):
    m, n, k = (1 << 20) + 4099, 16, 8192
    print("activations", m, n, k, flush=True)
    x, w = _random(wq, 1, m, k, 5), _random(wq, 1, n, k, 6)
    y = wq.wq_gemm_mx(x, w)
    wv = _values(w, slice(None))
    for rows in (slice(0, 64), slice((1 << 19) - 32, (1 << 19) + 32), slice((1 << 20) - 32, (1 << 20) + 32), slice(m - 64, m)):
        _check(y[rows], _values(x, rows), wv, k, "bf16", f"rows {rows}")


@pytest.mark.parametrize("t", [4, 300, 900])
def test_experts_beyond_4_gib(wq, t):
    """300 experts whose codes take 5 GB; only the last ones have rows: streaming and tiles."""
    import torch

    E, n, k = 300, 4096, 8192
    print("experts", t, E, n, k, flush=True)
    w = _random(wq, E, n, k, 7)
    cols = slice(n - 200, n)
    ids = np.where(np.arange(t) % 3 == 0, E - 2, E - 1).astype(np.int32)[:, None]
    off, order, _ = mx.route(ids, E)
    offsets, pairs = wq.wq_moe_route(torch.from_numpy(ids).cuda(), E)
    x = _random(wq, 1, t, k, 8)
    x.qscale -= 7  # the gate's sums of order 1
    h = wq.wq_moe_gate_up_mx(x, offsets, pairs, 1, w, w)
    d = wq.wq_moe_down_mx(x, offsets, w, dtype=torch.float32)
    xv = _values(x, slice(None))
    for e in (E - 2, E - 1):
        r = slice(int(off[e]), int(off[e + 1]))
        wv = _values(w, cols, e)
        g, gm = mx.product(xv[order[r]], wv)
        ref, bound = mx.gate_up_bound(g, gm, g, gm, k)
        mx.assert_within(mx.to_host(h[r, cols]), ref, bound, f"gate+up of expert {e}")
        _check(d[r, cols], xv[r], wv, k, "f32", f"down of expert {e}")


@pytest.mark.parametrize("t", [30, 260])
def test_512_experts(wq, t):
    import torch

    E, topk, n, k = 512, 8, 96, 320
    print("512 experts", t, flush=True)
    rng = np.random.default_rng(t)
    ids = rng.integers(0, E, (t, topk)).astype(np.int32)
    off, order, _ = mx.route(ids, E)
    offsets, pairs = wq.wq_moe_route(torch.from_numpy(ids).cuda(), E)
    w, x = _random(wq, E, n, k, 9), _random(wq, 1, t * topk, k, 10)
    d = wq.wq_moe_down_mx(x, offsets, w)
    tok = _random(wq, 1, t, k, 11)
    h = wq.wq_moe_gate_up_mx(tok, offsets, pairs, topk, w, w)
    xv, tv, dh, hh = _values(x, slice(None)), _values(tok, slice(None)), mx.to_host(d), mx.to_host(h)
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if off[e] == off[e + 1]:
            continue
        wv = _values(w, slice(None), e)
        ref, mag = mx.product(xv[r], wv)
        mx.assert_within(dh[r], ref, mx.sum_bound(ref, mag, k, "bf16"), f"down {e}")
        g, gm = mx.product(tv[order[r] // topk], wv)
        mx.assert_within(hh[r], *mx.gate_up_bound(g, gm, g, gm, k), f"gate+up {e}")


def test_nothing(wq):
    import torch

    E, n, k, topk = 4, 64, 128, 2
    w = _random(wq, E, n, k, 12)
    ids = torch.empty((0, topk), dtype=torch.int32, device="cuda")
    offsets, pairs = wq.wq_moe_route(ids, E)
    assert offsets.tolist() == [0] * (E + 1)
    x = wq.wq_quantize_mx(torch.empty((0, k), dtype=torch.bfloat16, device="cuda"))
    assert wq.wq_moe_gate_up_mx(x, offsets, pairs, topk, w, w).shape == (0, n)
    assert wq.wq_moe_down_mx(x, offsets, w).shape == (0, n)
    positions = wq.wq_moe_positions(ids, offsets, pairs)
    tokens = torch.empty((0, k), device="cuda")
    rows = wq.wq_moe_permute(tokens, positions)
    assert rows.shape == (0, k) and wq.wq_moe_unpermute(rows, positions).shape == (0, k)
    d_rows, d_w = wq.wq_moe_unpermute_grad(tokens, rows, positions)
    assert d_rows.shape == (0, k) and d_w.shape == (0, topk)
