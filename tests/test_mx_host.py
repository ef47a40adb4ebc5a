"""CPU tests of the MXFP4 calls and the token dispatch: refusals before any launch (none of these
calls reaches the GPU), layouts, and the test suite's own 64-bit encoder on printed values."""
import ctypes

import numpy as np
import pytest

import mx_testutil as mx
from test_abi import _weight, wq  # noqa: F401  (fixture)

P = [ctypes.c_void_p(0x10000 * (i + 1)) for i in range(9)]
ODD = ctypes.c_void_p(0x10008)


def _mx(wq, **kw):
    return _weight(wq, **{**dict(format=7, group=32, super_scale=None, code_scale=None, code_zero=None), **kw})


def test_encoder_of_the_tests_on_listed_values():
    # 32 values under a largest of 6 = 1.5 * 4: scale 1, the codes of the halves between neighbours
    v = np.zeros(32)
    v[:16] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.26, -0.74, 0.0, -0.0, 5.01, 2.49, 0.24, -6]
    code, byte = mx.encode(v)
    assert byte.tolist() == [127]
    assert code[:16].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 9, 9, 0, 8, 7, 4, 0, 15]
    code, byte = mx.encode(np.full(32, 7.99))  # below 8: the same scale, saturated
    assert byte.tolist() == [127] and set(code) == {7}
    assert mx.encode(np.full(32, 8.0))[1].tolist() == [128]
    assert mx.encode(np.zeros(32))[1].tolist() == [0]
    assert mx.encode(np.full(32, np.inf))[1].tolist() == [255]
    assert np.array_equal(mx.unpack(mx.pack(code[None])), code[None])


def test_layout(wq):
    assert wq._layout(wq.FMT_MXFP4, 2, 8, 128, 32) == {"codes": (2 * 8 * 64, 1), "qscale": (2 * 8 * 4, 1)}
    assert wq._layout(wq.FMT_MXFP4, 2, 8, 128, 64) is None
    assert wq._layout(wq.FMT_MXFP4, 2, 8, 96, 32) is None


@pytest.mark.parametrize("kw,status", [
    (dict(group=64), -2), (dict(group=0), -2), (dict(k=96), -2), (dict(qscale=None), -1),
    (dict(qscale=0x2008), -3), (dict(codes=None), -1), (dict(codes=0x1004), -3), (dict(n=0), -1),
    (dict(experts=3), -1), (dict(format=1, group=64, scales=0x6000), -2), (dict(n=1, k=1 << 30), -2),
    (dict(n=1 << 21, k=4096), -2),  # one expert's codes beyond the 32-bit range
])
def test_gemm_mx_rejects_bad_weights(wq, kw, status):
    L = wq.lib()
    w = _mx(wq, **kw)
    assert L.wq_gemm_mx(P[0], P[1], 4, ctypes.byref(w), P[2], 0, None) == status, L.wq_last_error()


@pytest.mark.parametrize("kw,status", [(dict(group=64), -2), (dict(qscale=None), -1), (dict(k=96), -2)])
def test_bf16_products_reject_bad_mxfp4(wq, kw, status):
    L = wq.lib()
    w = _mx(wq, **kw)
    assert L.wq_gemm(P[0], 4, ctypes.byref(w), P[2], None) == status
    assert L.wq_dequantize(ctypes.byref(w), P[2], None) == status


def test_gemm_mx_arguments(wq):
    L = wq.lib()
    w = ctypes.byref(_mx(wq))
    assert L.wq_gemm_mx(None, None, 0, w, None, 0, None) == 0
    assert L.wq_gemm_mx(P[0], P[1], -1, w, P[2], 0, None) == -1
    assert L.wq_gemm_mx(P[0], P[1], (1 << 31) + 1, w, P[2], 0, None) == -2
    assert L.wq_gemm_mx(P[0], P[1], 4, w, P[2], 2, None) == -2
    for bad, st in ((None, -1), (ODD, -3)):
        assert L.wq_gemm_mx(bad, P[1], 4, w, P[2], 0, None) == st
        assert L.wq_gemm_mx(P[0], bad, 4, w, P[2], 0, None) == st
        assert L.wq_gemm_mx(P[0], P[1], 4, w, bad, 1, None) == st
    assert L.wq_gemm_mx(P[0], P[1], 4, None, P[2], 0, None) == -1


def test_quantize_mx_arguments(wq):
    L = wq.lib()
    f = lambda x=P[0], t=0, n=4, k=64, c=P[1], s=P[2]: L.wq_quantize_mx(x, t, n, k, c, s, None)
    assert f(n=0, x=None) == 0
    assert f(t=2) == -2 and f(n=-1) == -1 and f(k=0) == -1 and f(k=96) == -2 and f(n=1 << 40) == -2
    for kw in ("x", "c", "s"):
        assert f(**{kw: None}) == -1 and f(**{kw: ODD}) == -3


def test_moe_mx_arguments(wq):
    L = wq.lib()
    g, u, d = _mx(wq, experts=4, n=128), _mx(wq, experts=4, n=128), _mx(wq, experts=4, n=256, k=128)
    up = lambda t=8, topk=2, gg=g, uu=u, a=P[:5]: L.wq_moe_gate_up_mx(a[0], a[1], t, a[2], a[3], topk, ctypes.byref(gg),
                                                                    ctypes.byref(uu), a[4], None)
    down = lambda n=16, dd=d, ty=0, a=P[:4]: L.wq_moe_down_mx(a[0], a[1], n, a[2], ctypes.byref(dd), a[3], ty, None)
    assert up(t=0, a=[None] * 5) == 0 and down(n=0, a=[None] * 4) == 0
    assert up(t=-1) == -1 and up(topk=0) == -1 and up(t=1 << 30) == -2 and down(n=-1) == -1 and down(ty=7) == -2
    assert up(uu=_mx(wq, experts=4, n=64)) == -1 and up(uu=_mx(wq, experts=5, n=128)) == -1
    assert up(gg=_mx(wq, experts=600, n=128), uu=_mx(wq, experts=600, n=128)) == -2
    other = _weight(wq, experts=4, n=128)  # CCQ experts: not this product's format
    assert up(gg=other, uu=other) == -2 and down(dd=_weight(wq, experts=4, n=256, k=128)) == -2
    for i in range(5):
        assert up(a=[None if j == i else P[j] for j in range(5)]) == -1
    for i in (0, 1, 4):
        assert up(a=[ODD if j == i else P[j] for j in range(5)]) == -3
    for i in range(4):
        assert down(a=[None if j == i else P[j] for j in range(4)]) == -1
    for i in (0, 1, 3):
        assert down(a=[ODD if j == i else P[j] for j in range(4)]) == -3


def test_dispatch_arguments(wq):
    L = wq.lib()
    pos = lambda t=4, k=2, e=8, a=P[:4]: L.wq_moe_positions(a[0], t, k, e, a[1], a[2], a[3], None)
    per = lambda ty=0, t=4, k=2, h=64, a=P[:3]: L.wq_moe_permute(a[0], ty, t, k, h, a[1], a[2], None)
    unp = lambda ty=0, t=4, k=2, h=64, a=P[:4]: L.wq_moe_unpermute(a[0], ty, a[1], a[2], t, k, h, a[3], None)
    grd = lambda ty=0, t=4, k=2, h=64, a=P[:6]: L.wq_moe_unpermute_grad(a[0], ty, a[1], a[2], a[3], t, k, h, a[4], a[5], None)
    assert pos(t=0, a=[None] * 4) == 0 and pos(e=0) == -1 and pos(e=513) == -2 and pos(k=0) == -1 and pos(t=1 << 30) == -2
    for i in range(4):
        assert pos(a=[None if j == i else P[j] for j in range(4)]) == -1
    for f, need, aligned in ((per, (0, 1, 2), (0, 2)), (unp, (0, 1, 3), (0, 3)), (grd, (0, 1, 2), (0, 1, 4))):
        n = max(need + aligned) + 1 if f is not grd else 6
        assert f(ty=5) == -2 and f(t=-1) == -1 and f(k=0) == -1 and f(h=0) == -1 and f(t=1 << 30) == -2
        assert f(h=(1 << 31) + 1) == -2
        assert f(t=0, a=[None] * n) == 0
        for i in need:
            assert f(a=[None if j == i else P[j] for j in range(n)]) == -1
        for i in aligned:
            assert f(a=[ODD if j == i else P[j] for j in range(n)]) == -3
    assert grd(a=[P[0], P[1], P[2], P[3], None, None]) == 0  # nothing asked for


def test_binding_refuses_host_and_wrong_tensors(wq):
    import torch

    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU tensor"):
        wq.wq_quantize_mx(x)
    with pytest.raises(TypeError, match="neither bf16 nor f32"):
        wq.wq_quantize_mx(x.half())
    with pytest.raises(TypeError, match="torch tensor"):
        wq.wq_quantize_mx(np.zeros((2, 64)))
    with pytest.raises(ValueError, match="multiple of 64"):
        wq.wq_quantize_mx(torch.zeros((2, 96)))
    with pytest.raises(ValueError, match=r"\[n, k\]"):
        wq.wq_quantize_mx(torch.zeros(64))
    w = wq.PackedWeight(wq.FMT_MXFP4, 8, 64, 1, 32, codes=torch.zeros((1, 8, 32), dtype=torch.uint8),
                        qscale=torch.zeros((1, 8, 2), dtype=torch.uint8))
    with pytest.raises(TypeError, match="PackedWeight"):
        wq.wq_gemm_mx(x, w)
    with pytest.raises(ValueError, match="GPU tensor"):
        wq.wq_gemm_mx(w, w)
    ids = torch.zeros((2, 2), dtype=torch.int32)
    for call in (lambda: wq.wq_moe_positions(ids, ids, ids), lambda: wq.wq_moe_permute(x, ids),
                 lambda: wq.wq_moe_unpermute(x, ids), lambda: wq.wq_moe_unpermute_grad(x, x, ids)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
