"""CPU tests of the int8 products, the norm and the balance loss: refusals before any launch (none of these
calls reaches the GPU), overlaps, the rules that choose a kernel, and the test suite's own definitions."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import i8_testutil as i8
from i8_cases import DENSE, EXPERTS, KERNELS, heights_of_last_tiles
from test_abi import _weight, wq  # noqa: F401  (fixture)

P = [ctypes.c_void_p(0x100000000 * (i + 1)) for i in range(9)]
ODD = ctypes.c_void_p(0x10008)
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_bit_amd", "csrc")


def _i8(wq, **kw):
    return _weight(wq, **{**dict(format=6, group=0, scales=0x20000, qscale=None, super_scale=None, code_scale=None,
                                 code_zero=None), **kw})


def test_definitions_on_listed_values():
    codes, a = i8.quantize([[127, 63.5, -0.5, 0.5, 1.5], [254, 127, 1, -3, 0], [0, 0, 0, 0, 0], [1, np.inf, 0, 0, 0]])
    assert codes.tolist() == [[127, 64, 0, 0, 2], [127, 64, 0, -2, 0], [0] * 5, [0] * 5]  # half way to even
    assert a[:3].tolist() == [127, 254, 0] and np.isnan(a[3])
    # half of the largest is half way between 63 and 64 whatever the largest
    assert all(i8.quantize([[v, v / 2]])[0].tolist() == [[127, 64]] for v in (1.0, 3.0, 0.1953125, 77.0))
    loss, counts, d, _, _ = i8.balance(np.zeros((3, 2)), np.array([[0], [0], [5]]), 0.5)
    assert loss == 0.5 and counts.tolist() == [2, 0, 2]  # p = 1/2: shares 2 and 0
    assert np.allclose(d, [[0.125, -0.125], [0.125, -0.125], [0, 0]])


def test_gradients_of_the_definitions_against_differences():
    rng = np.random.default_rng(0)
    r, w, dy, ds = rng.standard_normal((4, 3, 17))
    w = w[0]
    dx, dw = i8.norm_grad(dy, r, w, 1e-3, ds)
    h = 1e-5
    f = lambda r, w: (i8.norm(r, w, 1e-3)[0] * dy).sum() + (r * ds).sum()
    for _ in range(5):
        u, v = rng.standard_normal(r.shape), rng.standard_normal(w.shape)
        assert abs((f(r + h * u, w) - f(r - h * u, w)) / (2 * h) - (dx * u).sum()) < 1e-7
        assert abs((f(r, w + h * v) - f(r, w - h * v)) / (2 * h) - (dw * v).sum()) < 1e-7
    z, ids = rng.standard_normal((6, 5)), rng.integers(-1, 6, (6, 2))
    ids[2] = -1
    loss, counts, d, _, _ = i8.balance(z, ids, 0.3)
    for _ in range(5):
        u = rng.standard_normal(z.shape)
        diff = (i8.balance(z + h * u, ids, 0.3)[0] - i8.balance(z - h * u, ids, 0.3)[0]) / (2 * h)
        assert abs(diff - (d * u).sum()) < 1e-8


# ---------------------------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("kw,status", [
    (dict(group=64), -2), (dict(group=32), -2), (dict(k=96), -2), (dict(scales=None), -1), (dict(scales=0x2008), -3),
    (dict(codes=None), -1), (dict(codes=0x1004), -3), (dict(n=0), -1), (dict(experts=3), -1),
    (dict(format=1), -2), (dict(format=7, group=32, qscale=0x6000), -2),
    (dict(k=131072), -2),            # a sum of 128 * 128 over k could leave int32
    (dict(n=1 << 20, k=4096), -2),   # one expert's codes beyond the 32-bit range
])
def test_gemm_rejects_bad_weights(wq, kw, status):
    L = wq.lib()
    w = _i8(wq, **kw)
    assert L.wq_gemm_i8(P[0], P[1], 4, ctypes.byref(w), P[2], 0, None) == status, L.wq_last_error()
    assert L.wq_last_error()


def test_gemm_arguments(wq):
    L = wq.lib()
    w = ctypes.byref(_i8(wq))
    assert L.wq_gemm_i8(None, None, 0, w, None, 0, None) == 0
    assert L.wq_gemm_i8(None, None, 0, ctypes.byref(_i8(wq, k=131008)), None, 0, None) == 0  # the largest k
    assert L.wq_gemm_i8(P[0], P[1], -1, w, P[2], 0, None) == -1
    assert L.wq_gemm_i8(P[0], P[1], (1 << 31) + 1, w, P[2], 0, None) == -2
    assert L.wq_gemm_i8(P[0], P[1], 4, w, P[2], 2, None) == -2
    assert L.wq_gemm_i8(P[0], P[1], 4, None, P[2], 0, None) == -1
    assert [L.wq_gemm_i8(*a[:2], 4, w, a[2], 0, None) for a in ((None, P[1], P[2]), (P[0], None, P[2]), (P[0], P[1], None))] == [-1] * 3
    assert [L.wq_gemm_i8(*a[:2], 4, w, a[2], 0, None) for a in ((ODD, P[1], P[2]), (P[0], P[1], ODD))] == [-3] * 2


def test_moe_arguments(wq):
    L = wq.lib()
    g, u, d = _i8(wq, experts=4, n=128), _i8(wq, experts=4, n=128), _i8(wq, experts=4, n=256, k=128)
    up = lambda t=8, topk=2, gg=g, uu=u, a=P[:5]: L.wq_moe_gate_up_i8(a[0], a[1], t, a[2], a[3], topk, ctypes.byref(gg),
                                                                    ctypes.byref(uu), a[4], None)
    down = lambda n=16, dd=d, ty=0, a=P[:4]: L.wq_moe_down_i8(a[0], a[1], n, a[2], ctypes.byref(dd), a[3], ty, None)
    assert up(t=0, a=[None] * 5) == 0 and down(n=0, a=[None] * 4) == 0
    assert up(t=-1) == -1 and up(topk=0) == -1 and up(t=1 << 30) == -2 and down(n=-1) == -1 and down(ty=7) == -2
    assert up(uu=_i8(wq, experts=4, n=64)) == -1 and up(uu=_i8(wq, experts=5, n=128)) == -1
    assert up(gg=_i8(wq, experts=600, n=128), uu=_i8(wq, experts=600, n=128)) == -2
    group64 = _i8(wq, experts=4, n=128, group=64)
    assert up(gg=group64, uu=group64) == -2 and up(uu=group64) == -2
    assert up(uu=_i8(wq, experts=4, n=128, scales=None)) == -1 and up(uu=_i8(wq, experts=4, n=128, scales=0x2002)) == -3
    assert down(dd=_weight(wq, experts=4, n=256, k=128)) == -2
    for i in range(5):
        assert up(a=[None if j == i else P[j] for j in range(5)]) == -1
    for i in (0, 4):
        assert up(a=[ODD if j == i else P[j] for j in range(5)]) == -3
    for i in range(4):
        assert down(a=[None if j == i else P[j] for j in range(4)]) == -1
    for i in (0, 3):
        assert down(a=[ODD if j == i else P[j] for j in range(4)]) == -3


def test_quantize_arguments(wq):
    L = wq.lib()
    f = lambda x=P[0], t=0, n=4, k=65, c=P[1], s=P[2], st=1: L.wq_quantize_i8(x, t, n, k, c, s, st, None)
    assert f(n=0, x=None) == 0
    assert f(t=2) == -2 and f(st=3) == -2 and f(n=-1) == -1 and f(k=0) == -1 and f(n=1 << 40) == -2
    for kw in ("x", "c", "s"):
        assert f(**{kw: None}) == -1
    assert f(x=ODD) == -3 and f(c=ODD) == -3


def test_norm_arguments(wq):
    L = wq.lib()
    base = dict(x=P[0], ty=0, res=P[1], w=P[2], eps=1e-6, n=4, k=65, sum=P[3], y=P[4], s=P[5])
    plain = lambda **kw: (lambda a: L.wq_rms_norm(a["x"], a["ty"], a["res"], a["w"], a["eps"], a["n"], a["k"], a["sum"],
                                                  a["y"], None))({**base, **kw})
    codes = lambda **kw: (lambda a: L.wq_rms_norm_i8(a["x"], a["ty"], a["res"], a["w"], a["eps"], a["n"], a["k"],
                                                     a["sum"], a["y"], a["s"], None))({**base, **kw})
    for f in (plain, codes):
        assert f(n=0, x=None, res=None, sum=None, y=None, w=None) == 0
        assert f(ty=2) == -2 and f(n=-1) == -1 and f(k=0) == -1 and f(n=1 << 40) == -2
        for eps in (-1e-6, float("nan"), float("inf")):
            assert f(eps=eps) == -1
        for kw in ("x", "w", "y"):
            assert f(**{kw: None}) == -1
        for kw in ("x", "res", "w", "sum", "y"):
            assert f(**{kw: ODD}) == -3
        assert f(res=None) == -1 and f(sum=None) == -1  # together, or neither
    assert codes(s=None) == -1


def test_norm_grad_arguments(wq):
    L = wq.lib()
    base = dict(dy=P[0], ty=0, ds=P[1], sum=P[2], w=P[3], eps=1e-6, n=400, k=65, dx=P[4], dw=P[5], ws=P[6], b=None)

    def f(**kw):
        a = {**base, **kw}
        b = L.wq_rms_norm_grad_workspace_bytes(a["n"], a["k"], a["ty"]) if a["b"] is None else a["b"]
        return L.wq_rms_norm_grad(a["dy"], a["ty"], a["ds"], a["sum"], a["w"], a["eps"], a["n"], a["k"], a["dx"], a["dw"],
                                  a["ws"], b, None)

    need = L.wq_rms_norm_grad_workspace_bytes(400, 65, 0)
    assert need > 0 and need % (65 * 4) == 0
    assert L.wq_rms_norm_grad_workspace_bytes(1, 65, 0) == 0  # one row's products are the gradient
    assert [L.wq_rms_norm_grad_workspace_bytes(*a) for a in ((-1, 65, 0), (4, 0, 0), (4, 65, 2), (1 << 40, 65, 0))] == [0] * 4
    assert f(ty=2) == -2 and f(n=-1, b=0, ws=None) == -1 and f(k=0, b=0) == -1 and f(eps=-1.0) == -1
    assert f(b=need - 1) == -5 and f(ws=None, b=0) == -5 and f(ws=None) == -1
    assert f(n=0, dw=None, dy=None, sum=None, w=None, dx=None) == 0
    for kw in ("dy", "sum", "w", "dx"):
        assert f(**{kw: None}) == -1
    for kw in ("dy", "ds", "sum", "w", "dx", "dw", "ws"):
        assert f(**{kw: ODD}) == -3


def test_balance_arguments(wq):
    L = wq.lib()
    base = dict(z=P[0], ty=0, ids=P[1], t=4096, topk=2, E=60, loss=P[2], c=P[3], ws=P[4], b=None, d=P[5], dl=P[6])

    def f(**kw):
        a = {**base, **kw}
        b = L.wq_moe_balance_loss_workspace_bytes(a["t"], a["E"]) if a["b"] is None else a["b"]
        return L.wq_moe_balance_loss(a["z"], a["ty"], a["ids"], a["t"], a["topk"], a["E"], 1.0, a["loss"], a["c"], a["ws"],
                                     b, None)

    def g(**kw):
        a = {**base, **kw}
        return L.wq_moe_balance_loss_grad(a["z"], a["ty"], a["ids"], a["t"], a["topk"], a["E"], 1.0, a["c"], a["dl"],
                                          a["d"], None)

    need = L.wq_moe_balance_loss_workspace_bytes(4096, 60)
    assert need > 0 and L.wq_moe_balance_loss_workspace_bytes(1, 60) == 0
    assert [L.wq_moe_balance_loss_workspace_bytes(*a) for a in ((-1, 60), (4096, 0), (4096, 513), ((1 << 30) + 1, 60))] == [0] * 4
    assert f(b=need - 1) == -5 and f(ws=None, b=0) == -5 and f(ws=None) == -1
    for h in (f, g):
        assert h(ty=2) == -2 and h(t=-1, b=0, ws=None) == -1 and h(topk=0) == -1 and h(E=0, b=0, ws=None) == -1
        assert h(E=513, b=0, ws=None) == -2 and h(t=1 << 30, b=0, ws=None) == -2
        assert h(z=None) == -1 and h(ids=None) == -1 and h(c=None) == -1 and h(z=ODD) == -3
    assert f(loss=None) == -1 and f(ws=ODD) == -3 and g(d=None) == -1 and g(d=ODD) == -3
    assert g(t=0, z=None, ids=None, c=None, d=None) == 0


def test_binding_refuses_host_and_wrong_tensors(wq):
    import torch

    x, w = torch.zeros((2, 64), dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    ids = torch.zeros((2, 2), dtype=torch.int32)
    pw = wq.PackedWeight(wq.FMT_INT8, 8, 64, 1, 0, codes=torch.zeros((1, 8, 64), dtype=torch.int8),
                         scales=torch.zeros((1, 8), dtype=torch.bfloat16))
    rows = wq.Int8Rows(torch.zeros((2, 64), dtype=torch.int8), torch.zeros(2))
    for call in (lambda: wq.wq_quantize_i8(x), lambda: wq.wq_quantize_i8_weight(x), lambda: wq.wq_gemm_i8(rows, pw),
                 lambda: wq.wq_moe_gate_up_i8(rows, ids, ids, 2, pw, pw), lambda: wq.wq_moe_down_i8(rows, ids, pw),
                 lambda: wq.wq_rms_norm(x, w), lambda: wq.wq_rms_norm_i8(x, w, x), lambda: wq.wq_rms_norm_grad(x, x, w),
                 lambda: wq.wq_moe_balance_loss(x, ids), lambda: wq.wq_moe_balance_loss_grad(x, ids, ids)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(TypeError, match="neither bf16 nor f32"):
        wq.wq_quantize_i8(x.half())
    with pytest.raises(TypeError, match="neither bf16 nor f32"):
        wq.wq_rms_norm(x.half(), w)
    with pytest.raises(TypeError, match="torch tensor"):
        wq.wq_moe_balance_loss(np.zeros((2, 64)), ids)
    with pytest.raises(TypeError, match="Int8Rows"):
        wq.wq_gemm_i8(x, pw)
    with pytest.raises(ValueError, match=r"\[n, k\]"):
        wq.wq_quantize_i8(torch.zeros(64))
    with pytest.raises(ValueError, match="multiple of 64"):
        wq.wq_quantize_i8_weight(torch.zeros((2, 96)))
    with pytest.raises(ValueError, match=r"\[t, topk\]"):
        wq.wq_moe_balance_loss(x, ids[0])


# ---------------------------------------------------------------------------------------------
# overlaps: every output at three places of every other array (its first byte, its last 16, and so that the
# output's own last 16 bytes lie on the array's first ones)
# ---------------------------------------------------------------------------------------------

FAR = 1 << 32


def _calls(wq):
    """name -> (bytes of every array, outputs, pairs (output, input) that may share their address, call)."""
    L, ref = wq.lib(), ctypes.byref
    E, n, k, m, t, topk = 3, 48, 128, 700, 5000, 2
    pairs = 60

    def w8(e, a, codes="codes", scales="scales"):
        return _i8(wq, experts=e, n=n, k=k, codes=a[codes], scales=a[scales])

    out = {}
    for ty, size in ((0, 2), (1, 4)):
        for st, ss in ((0, 2), (1, 4)):
            out[f"quantize {ty} {st}"] = ({"x": m * k * size, "codes": m * k, "scales": m * ss}, ("codes", "scales"), (),
                lambda a, ty=ty, st=st: L.wq_quantize_i8(a["x"], ty, m, k, a["codes"], a["scales"], st, None))
        out[f"gemm {ty}"] = ({"xc": m * k, "xs": m * 4, "codes": n * k, "scales": n * 2, "y": m * n * size}, ("y",), (),
            lambda a, ty=ty: L.wq_gemm_i8(a["xc"], a["xs"], m, ref(w8(1, a)), a["y"], ty, None))
        out[f"down {ty}"] = (
            {"hc": pairs * k, "hs": pairs * 4, "codes": E * n * k, "scales": E * n * 2, "off": 4 * (E + 1),
             "d": pairs * n * size}, ("d",), (),
            lambda a, ty=ty: L.wq_moe_down_i8(a["hc"], a["hs"], pairs, a["off"], ref(w8(E, a)), a["d"], ty, None))
        v = m * k * size
        out[f"norm {ty}"] = ({"x": v, "res": v, "w": k * size, "sum": v, "y": v}, ("sum", "y"),
                             (("sum", "x"), ("sum", "res")),
            lambda a, ty=ty: L.wq_rms_norm(a["x"], ty, a["res"], a["w"], 1e-6, m, k, a["sum"], a["y"], None))
        out[f"norm_i8 {ty}"] = ({"x": v, "res": v, "w": k * size, "sum": v, "codes": m * k, "scales": m * 4},
                                ("sum", "codes", "scales"), (("sum", "x"), ("sum", "res")),
            lambda a, ty=ty: L.wq_rms_norm_i8(a["x"], ty, a["res"], a["w"], 1e-6, m, k, a["sum"], a["codes"], a["scales"], None))
        need = L.wq_rms_norm_grad_workspace_bytes(m, k, ty)
        out[f"norm_grad {ty}"] = ({"dy": v, "ds": v, "sum": v, "w": k * size, "dx": v, "dw": k * 4, "ws": need},
                                  ("dx", "dw", "ws"), (("dx", "ds"),),
            lambda a, ty=ty, need=need: L.wq_rms_norm_grad(a["dy"], ty, a["ds"], a["sum"], a["w"], 1e-6, m, k, a["dx"], a["dw"],
                                                           a["ws"], need, None))
        z, need = t * E * size, L.wq_moe_balance_loss_workspace_bytes(t, E)
        assert need
        out[f"balance {ty}"] = ({"z": z, "ids": t * topk * 4, "loss": 4, "counts": 4 * (E + 1), "ws": need},
                                ("loss", "counts", "ws"), (),
            lambda a, ty=ty, need=need: L.wq_moe_balance_loss(a["z"], ty, a["ids"], t, topk, E, 1.0, a["loss"], a["counts"],
                                                              a["ws"], need, None))
        out[f"balance_grad {ty}"] = ({"z": z, "ids": t * topk * 4, "counts": 4 * (E + 1), "dl": 4, "d": z}, ("d",), (),
            lambda a, ty=ty: L.wq_moe_balance_loss_grad(a["z"], ty, a["ids"], t, topk, E, 1.0, a["counts"], a["dl"], a["d"], None))
    tok = 30
    out["gate_up"] = (
        {"xc": tok * k, "xs": tok * 4, "off": 4 * (E + 1), "pairs": 4 * pairs, "codes": E * n * k, "scales": E * n * 2,
         "up_codes": E * n * k, "up_scales": E * n * 2, "h": pairs * n * 2}, ("h",), (),
        lambda a: L.wq_moe_gate_up_i8(a["xc"], a["xs"], tok, a["off"], a["pairs"], 2, ref(w8(E, a)),
                                      ref(w8(E, a, "up_codes", "up_scales")), a["h"], None))
    return out


NAMES = [f"{c} {ty}" for ty in (0, 1) for c in ("gemm", "down", "norm", "norm_i8", "norm_grad", "balance", "balance_grad")]
NAMES += [f"quantize {ty} {st}" for ty in (0, 1) for st in (0, 1)] + ["gate_up"]


@pytest.mark.parametrize("name", NAMES)
def test_overlaps_are_refused(wq, name):
    sizes, outputs, shared, call = _calls(wq)[name]
    at = {a: FAR * (i + 1) for i, a in enumerate(sizes)}
    tried = 0
    for o in outputs:
        for other in sizes:
            if other == o:
                continue
            last = (sizes[other] - 1) // 16 * 16
            for i, place in enumerate((at[other], at[other] + last, at[other] - (sizes[o] - 1) // 16 * 16)):
                if place == at[other] and (o, other) in shared:
                    continue
                st = call({**at, o: place})
                assert st == -1, (o, other, i)
                assert "overlap" in wq.lib().wq_last_error().decode(), (o, other)
                tried += 1
    assert tried >= 2 * len(outputs)


def test_every_call_is_listed(wq):
    assert sorted(_calls(wq)) == sorted(NAMES)


# ---------------------------------------------------------------------------------------------
# which kernel a product takes (csrc/wq_i8_select.hpp, compiled here for the CPU)
# ---------------------------------------------------------------------------------------------

SOURCE = """
#include "wq_i8_select.hpp"
extern "C" int dense(int64_t m, int64_t n, int64_t k) { return wq::i8_dense_kernel(m, n, k); }
extern "C" int experts(int64_t gathered, int64_t pairs, int64_t n, int64_t k, int64_t e) {
  return wq::i8_experts_kernel(gathered, pairs, n, k, e);
}
extern "C" int number(int i) {
  constexpr wq::I8Kernel names[] = {NAMES};
  return names[i];
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    d = tmp_path_factory.mktemp("select")
    src, so = d / "select.cpp", d / "select.so"
    src.write_text(SOURCE.replace("NAMES", ", ".join("wq::" + k for k in KERNELS)))
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", f"-I{CSRC}", str(src), "-o", str(so)],
                   check=True)
    L = ctypes.CDLL(str(so))
    for f, n in ((L.dense, 3), (L.experts, 5)):
        f.argtypes = [ctypes.c_int64] * n
    assert [L.number(i) for i in range(len(KERNELS))] == list(range(len(KERNELS)))
    return L


def _height(kernel):
    return {"I8_TILES_256": 256, "I8_TILES_64": 64}.get(kernel, 128)


def test_cases_take_their_kernels(rules):
    for c in DENSE:
        assert KERNELS[rules.dense(c.m, c.n, c.k)] == c.kernel, c
    assert {c.kernel for c in DENSE} == set(KERNELS)
    for c in EXPERTS:
        assert sum(c.counts) <= c.t * c.topk
        got = KERNELS[rules.experts(c.t if c.gate_up else 0, c.t * c.topk, c.n, c.k, len(c.counts))]
        assert got == c.kernel, (c, got)
    groups = [[(c.kernel, [c.m], c.k) for c in DENSE]]
    groups += [[(c.kernel, c.counts, c.k) for c in EXPERTS if c.gate_up == up] for up in (True, False)]
    for i, group in enumerate(groups):
        kernels = {g[0] for g in group}
        if i:
            assert kernels == {"I8_STREAM_16", "I8_TILES_128", "I8_TILES_128x256", "I8_TILES_256"}, i
        for kernel in kernels:
            if "TILES" not in kernel:
                continue
            some = [g for g in group if g[0] == kernel]
            # every height of a last row tile, and a stage (128) that k ends inside
            heights = set().union(*(heights_of_last_tiles(g[1], _height(kernel)) for g in some))
            assert heights == set(range(1, _height(kernel) // 64 + 1)), (kernel, heights)
            assert any(g[2] % 128 for g in some), kernel


def test_limits_of_the_tiles(rules):
    dense = lambda *a: KERNELS[rules.dense(*a)]
    # one expert's codes: n k up to 2^31 - 1024
    assert dense(64, (1 << 20) - 1, 2048).startswith("I8_TILES") and dense(64, 1 << 20, 2048) == "I8_STREAM_32"
    assert dense(4096, 8192, 64) == "I8_TILES_256" and dense(16, 4096, 1024) == "I8_STREAM_16"
    # gate+up gathers its tokens from all of them: 262143 tokens of hidden 8192
    for t, tiles in ((262143, True), (262144, False)):
        assert (KERNELS[rules.experts(t, 8 * t, 3584, 8192, 64)] != "I8_STREAM_16") == tiles
        assert KERNELS[rules.experts(0, 8 * t, 8192, 3584, 64)] == "I8_TILES_256"
