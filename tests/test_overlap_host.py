"""MXFP4 quantisation, the products of two MXFP4 operands and the token dispatch refuse an output that
shares memory with any input, or with another output (CPU: nothing is launched).

Every call is made with its arrays far apart but for the output under test, which is put at three places of
one other array: on its first byte, over its last 16 bytes, and so that its own last 16 bytes lie on the
array's first ones."""
import ctypes
import os

import pytest

FAR = 1 << 32  # between arrays; none is as long


@pytest.fixture(scope="module")
def wq():
    import weight_only_bit_amd as wq

    if not os.path.exists(wq.LIB_PATH):
        from weight_only_bit_amd import build

        build.build()
    wq.lib()
    return wq


def _weight(wq, E, n, k, at):
    return wq._CWeight(wq.FMT_MXFP4, 32, E, n, k, at["codes"], None, None, at["scales"], None, None, None, 32)


def _calls(wq):
    """name -> (sizes in bytes of every array, outputs, call(addresses) -> status)."""
    L, ref = wq.lib(), ctypes.byref
    E, n, k, m, t, topk, h = 3, 48, 128, 5, 6, 2, 64
    P = t * topk
    out = {}
    for ty, size in ((0, 2), (1, 4)):
        out[f"quantize {ty}"] = ({"x": m * k * size, "codes": m * k // 2, "scales": m * k // 32}, ("codes", "scales"),
                                 lambda a, ty=ty: L.wq_quantize_mx(a["x"], ty, m, k, a["codes"], a["scales"], None))
        out[f"gemm {ty}"] = (
            {"xc": m * k // 2, "xs": m * k // 32, "codes": n * k // 2, "scales": n * k // 32, "y": m * n * size}, ("y",),
            lambda a, ty=ty: L.wq_gemm_mx(a["xc"], a["xs"], m, ref(_weight(wq, 1, n, k, a)), a["y"], ty, None))
        out[f"down {ty}"] = (
            {"hc": P * k // 2, "hs": P * k // 32, "codes": E * n * k // 2, "scales": E * n * k // 32, "off": 4 * (E + 1),
             "d": P * n * size}, ("d",),
            lambda a, ty=ty: L.wq_moe_down_mx(a["hc"], a["hs"], P, a["off"], ref(_weight(wq, E, n, k, a)), a["d"], ty, None))
        rows, tok = P * h * size, t * h * size
        out[f"permute {ty}"] = ({"x": tok, "pos": 4 * P, "rows": rows}, ("rows",),
                                lambda a, ty=ty: L.wq_moe_permute(a["x"], ty, t, topk, h, a["pos"], a["rows"], None))
        out[f"unpermute {ty}"] = (
            {"rows": rows, "pos": 4 * P, "w": 4 * P, "y": tok}, ("y",),
            lambda a, ty=ty: L.wq_moe_unpermute(a["rows"], ty, a["pos"], a["w"], t, topk, h, a["y"], None))
        out[f"unpermute_grad {ty}"] = (
            {"dy": tok, "rows": rows, "pos": 4 * P, "w": 4 * P, "d_rows": rows, "d_w": 4 * P}, ("d_rows", "d_w"),
            lambda a, ty=ty: L.wq_moe_unpermute_grad(a["dy"], ty, a["rows"], a["pos"], a["w"], t, topk, h, a["d_rows"],
                                                     a["d_w"], None))

    def gate_up(a):
        up = {"codes": a["up_codes"], "scales": a["up_scales"]}
        return L.wq_moe_gate_up_mx(a["xc"], a["xs"], t, a["off"], a["pairs"], topk, ref(_weight(wq, E, n, k, a)),
                                   ref(_weight(wq, E, n, k, up)), a["h"], None)

    w = {"codes": E * n * k // 2, "scales": E * n * k // 32}
    out["gate_up"] = ({"xc": t * k // 2, "xs": t * k // 32, "off": 4 * (E + 1), "pairs": 4 * P, **w,
                       "up_codes": w["codes"], "up_scales": w["scales"], "h": P * n * 2}, ("h",), gate_up)
    out["positions"] = ({"ids": 4 * P, "off": 4 * (E + 1), "pairs": 4 * P, "pos": 4 * P}, ("pos",),
                        lambda a: L.wq_moe_positions(a["ids"], t, topk, E, a["off"], a["pairs"], a["pos"], None))
    return out


NAMES = ["quantize 0", "quantize 1", "gemm 0", "gemm 1", "down 0", "down 1", "permute 0", "permute 1", "unpermute 0",
         "unpermute 1", "unpermute_grad 0", "unpermute_grad 1", "gate_up", "positions"]


@pytest.mark.parametrize("name", NAMES)
def test_overlaps_are_refused(wq, name):
    sizes, outputs, call = _calls(wq)[name]
    at = {a: FAR * (i + 1) for i, a in enumerate(sizes)}
    tried = 0
    for o in outputs:
        for other in sizes:
            if other == o:
                continue
            last = (sizes[other] - 1) // 16 * 16
            for place in (at[other], at[other] + last, at[other] - (sizes[o] - 1) // 16 * 16):
                st = call({**at, o: place})
                assert st == -1, (o, other, hex(place))
                assert "overlap" in wq.lib().wq_last_error().decode(), (o, other)
                tried += 1
    assert tried == 3 * len(outputs) * (len(sizes) - 1)


def test_every_call_is_listed(wq):
    assert sorted(_calls(wq)) == sorted(NAMES)
