"""Every kernel of the products of two MXFP4 operands (the cases of mx_cases.py, whose kernels
test_mx_select_host.py asserts), and the kernels with bf16 activations, against fp64: values, NaN blocks,
extreme scales, the same bits on every run and beside another stream.  Codes are drawn uniformly, scales over seven octaves; references and bounds (those
derived in mx_testutil, here in torch) are float64 on the GPU."""
import numpy as np
import pytest

import mx_testutil as mx
from mx_cases import DENSE, EXPERTS

pytestmark = pytest.mark.gpu

OUT = ("bf16", "f32")
# rows whose blocks hold NaN: a tile's first and last rows at every height, and the matrix's
EDGES = (0, 31, 32, 63, 64, 127, 128, 255, 256)


@pytest.fixture(scope="module")
def wq():
    import torch

    import weight_only_bit_amd as wq

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    wq.lib()
    yield wq
    torch.cuda.empty_cache()


def _name(c):
    return "-".join(str(v) for v in c).replace(" ", "")


class Mat:
    """MXFP4 values [E, n, k] on the GPU: uniform codes, scale bytes around `middle`."""

    def __init__(self, wq, g, E, n, k, middle=127):
        import torch

        self.wq, self.shape = wq, (E, n, k)
        self.code = torch.randint(0, 16, (E, n, k), generator=g, device="cuda", dtype=torch.uint8)
        self.byte = (torch.randint(-3, 4, (E, n, k // 32), generator=g, device="cuda") + middle).to(torch.uint8)

    def nan(self, e, row, block):
        """`row` and `block` from the end where negative; rows behind the end are left out."""
        if row < self.shape[1]:
            self.byte[e, row, block] = 255
        return self

    def packed(self):
        c = self.code
        E, n, k = self.shape
        return self.wq.PackedWeight(self.wq.FMT_MXFP4, n, k, E, 32, codes=c[..., 0::2] | (c[..., 1::2] << 4),
                                    qscale=self.byte)

    def values(self, e=0, rows=slice(None)):
        """fp64, NaN where the scale byte is 255."""
        import torch

        table = torch.tensor(mx.VALUES, dtype=torch.float64, device="cuda")
        b = self.byte[e, rows]
        scale = torch.where(b == 255, float("nan"), torch.exp2(b.double() - 127))
        return (table[self.code[e, rows].int()].view(*b.shape, 32) * scale.unsqueeze(-1)).view(b.shape[0], -1)


def _product(x, w):
    """(x w^T, sum of the products' magnitudes without the NaN ones)."""
    import torch

    wt = w.t().contiguous()
    return torch.mm(x, wt), torch.mm(x.nan_to_num().abs(), wt.nan_to_num().abs())


def _sum_bound(ref, mag, k, out):
    err = k * 2.0 ** -23 * mag
    return err + mx.HALF[out] * (ref.abs() + err) + 2.0 ** -133


def _gate_up_bound(g, gm, u, um, k):
    import torch

    dg, du = k * 2.0 ** -23 * gm, k * 2.0 ** -23 * um
    h = g / (1 + torch.exp(-g.clamp_min(-700))) * u
    err = 1.1 * dg * (u.abs() + du) + g.abs() * du + h.abs() * (8 + 2 * g.abs()) * 2.0 ** -23
    return h, err + mx.HALF["bf16"] * (h.abs() + err) + 2.0 ** -126


def _within(got, ref, bound, what):
    got = got.double()
    nan = ref.isnan()
    assert bool((got.isnan() == nan).all()), f"{what}: NaN at other places than expected"
    bad = ~nan & ~((got - ref).abs() <= bound)
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())}/{ref.numel()} outside; first at {i}: got {float(got[i])!r}, "
                             f"want {float(ref[i])!r}, bound {float(bound[i]):.3g}")


def _gen(seed):
    import torch

    return torch.Generator(device="cuda").manual_seed(seed)


def _out(torch, rows, n, out):
    return torch.full((rows, n), 9.0, dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")


@pytest.mark.parametrize("out", OUT)
@pytest.mark.parametrize("kind", ["values", "nan", "large weights", "small weights"])
@pytest.mark.parametrize("case", DENSE, ids=_name)
def test_dense(wq, case, kind, out):
    import torch

    print("dense", *case, kind, out, flush=True)
    m, n, k = case.m, case.n, case.k
    g = _gen(m + n)
    # weights near the largest and the least scales, activations the other way round
    wm, xm = {"large weights": (247, 7), "small weights": (7, 247)}.get(kind, (127, 127))
    w, x = Mat(wq, g, 1, n, k, wm), Mat(wq, g, 1, m, k, xm)
    if kind == "nan":
        for r in EDGES:
            w.nan(0, r, 0 if r % 2 else -1)
            x.nan(0, r, -1 if r % 2 else 0)
        w.nan(0, n - 1, -1)
        x.nan(0, m - 1, -1)
        w.nan(0, n // 2, k // 64)
        x.nan(0, m // 2, k // 64)
    y = _out(torch, m + 1, n, out)
    wq.wq_gemm_mx(x.packed(), w.packed(), y=y[:m])
    assert bool((y[m] == 9.0).all()), "the row behind the last one was written"
    ref, mag = _product(x.values(), w.values())
    _within(y[:m], ref, _sum_bound(ref, mag, k, out), f"{case} {kind}")


def _routing(torch, g, c):
    """(offsets, sorted pairs on the GPU; the token of every row): any order of the pairs will do."""
    P = c.t * c.topk
    off = np.concatenate([[0], np.cumsum(c.counts)]).astype(np.int32)
    pairs = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    return off, torch.from_numpy(off).cuda(), pairs, (pairs // c.topk).long()


@pytest.mark.parametrize("kind", ["values", "nan", "large weights", "small weights"])
@pytest.mark.parametrize("case,out", [(c, o) for c in EXPERTS for o in OUT if not (c.gate_up and o == "f32")],
                         ids=lambda v: v if isinstance(v, str) else _name(v))
def test_experts(wq, case, out, kind):
    import torch

    print("experts", *case, kind, out, flush=True)
    c, E, P, g = case, len(case.counts), case.t * case.topk, _gen(case.n)
    off, offsets, pairs, token = _routing(torch, g, c)
    # activations small enough that the gate's sums are of order 1
    wm, xm = {"large weights": (247, -1), "small weights": (7, 239)}.get(kind, (127, 119))
    xm = max(xm, 3)
    mats = [Mat(wq, g, E, c.n, c.k, wm) for _ in range(2 if c.gate_up else 1)]
    x = Mat(wq, g, 1, c.t if c.gate_up else P, c.k, xm)
    if kind == "nan":
        for e in range(E):  # an expert's own rows of both matrices
            for r in EDGES:
                mats[(r + e) % len(mats)].nan(e, r, 0 if (r + e) % 2 else -1)
            mats[-1].nan(e, c.n - 1, -1)
            if off[e + 1] > off[e] and not c.gate_up:
                for r in EDGES + (c.counts[e] - 1,):
                    if r < c.counts[e]:
                        x.nan(0, int(off[e]) + r, -1 if r % 2 else 0)
        if c.gate_up:
            for t in (0, 1, c.t // 2, c.t - 1):
                x.nan(0, t, -1 if t % 2 else 0)
    o = _out(torch, P, c.n, out)
    if c.gate_up:
        wq.wq_moe_gate_up_mx(x.packed(), offsets, pairs, c.topk, mats[0].packed(), mats[1].packed(), h=o)
    else:
        wq.wq_moe_down_mx(x.packed(), offsets, mats[0].packed(), d=o)
    assert bool((o[int(off[-1]):] == 9.0).all()), "rows behind the last expert's were written"
    for e in range(E):
        if off[e] == off[e + 1]:
            continue
        r = slice(int(off[e]), int(off[e + 1]))
        xe = x.values(0, token[r] if c.gate_up else r)
        a, am = _product(xe, mats[0].values(e))
        if c.gate_up:
            ref, bound = _gate_up_bound(a, am, *_product(xe, mats[1].values(e)), c.k)
        else:
            ref, bound = a, _sum_bound(a, am, c.k, out)
        _within(o[r], ref, bound, f"expert {e} of {case} {kind}")


def _repeat(torch, calls):
    """Every call alone five times, then all of them on streams of their own at once: the same bits."""
    first = [f() for f in calls]
    torch.cuda.synchronize()
    for f, want in zip(calls, first):
        for _ in range(5):
            assert torch.equal(f(), want)
    streams = [torch.cuda.Stream() for _ in calls]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for f, s, want in zip(calls, streams, first):
            with torch.cuda.stream(s):
                got.append((f(), want))
    torch.cuda.synchronize()
    for a, b in got:
        assert torch.equal(a, b)


@pytest.mark.parametrize("case", DENSE, ids=_name)
def test_dense_repeats(wq, case):
    import torch

    print("repeat", *case, flush=True)
    g = _gen(case.k)
    calls = []
    for i in range(2):
        w, x = Mat(wq, g, 1, case.n, case.k).packed(), Mat(wq, g, 1, case.m - 5 * i, case.k).packed()
        calls.append(lambda w=w, x=x: wq.wq_gemm_mx(x, w))
    _repeat(torch, calls)


@pytest.mark.parametrize("case", EXPERTS, ids=_name)
def test_experts_repeat(wq, case):
    import torch

    print("repeat", *case, flush=True)
    c, E, g = case, len(case.counts), _gen(case.k)
    off, offsets, pairs, _ = _routing(torch, g, c)
    P, live = c.t * c.topk, int(off[-1])
    calls = []
    for _ in range(2):
        ws = [Mat(wq, g, E, c.n, c.k).packed() for _ in range(2 if c.gate_up else 1)]
        x = Mat(wq, g, 1, c.t if c.gate_up else P, c.k, 119).packed()
        if c.gate_up:
            calls.append(lambda ws=ws, x=x: wq.wq_moe_gate_up_mx(x, offsets, pairs, c.topk, *ws)[:live])
        else:
            calls.append(lambda ws=ws, x=x: wq.wq_moe_down_mx(x, offsets, ws[0])[:live])
    _repeat(torch, calls)


# ---------------------------------------------------------------------------------------------
# bf16 activations: the single-staging (at most 16 rows) and decode-streaming kernels, and from 2.75 million
# outputs on (1.15 and 1.68 million for 64 and 128 rows) the tiled one; experts by 32 rows on average
# ---------------------------------------------------------------------------------------------

BF16_DENSE = [(5, 40, 1024), (24, 96, 4160), (300, 530, 704), (40, 28801, 192), (100, 17001, 64), (1400, 2001, 320),
              (700, 4000, 832)]
BF16_EXPERTS = [(20, 2, 65, 576, (0, 17, 1, 16, 3)), (12, 4, 128, 512, (6, 6, 6, 12, 0, 3, 9, 5)),
                (300, 2, 350, 704, (180, 326, 64)), (100, 4, 513, 320, (40, 0, 260))]
KINDS = ["values", "nan", "large weights", "small weights"]


def _middles(kind, x=127):
    return {"large weights": (247, 7), "small weights": (7, 247)}.get(kind, (127, x))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n,k", BF16_DENSE)
def test_dense_bf16_activations(wq, m, n, k, kind):
    import torch

    print("bf16 dense", m, n, k, kind, flush=True)
    g = _gen(m + n)
    wm, xm = _middles(kind)
    w, x = Mat(wq, g, 1, n, k, wm), Mat(wq, g, 1, m, k, xm)
    if kind == "nan":
        for r in EDGES:
            w.nan(0, r, 0 if r % 2 else -1)
        w.nan(0, n - 1, -1)
    xv, p = x.values(), w.packed()  # e2m1 values times powers of two are bf16 values
    y = _out(torch, m + 1, n, "bf16")
    xb = xv.to(torch.bfloat16)
    wq.wq_gemm(xb, p, y=y[:m])
    assert bool((y[m] == 9.0).all()), "the row behind the last one was written"
    ref, mag = _product(xv, w.values())
    _within(y[:m], ref, _sum_bound(ref, mag, k, "bf16"), f"{m} {n} {k} {kind}")
    if kind == "values":
        other = xb[: m - m // 3]
        _repeat(torch, [lambda: wq.wq_gemm(xb, p), lambda: wq.wq_gemm(other, p)])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t,topk,inter,hidden,counts", BF16_EXPERTS)
def test_experts_bf16_activations(wq, t, topk, inter, hidden, counts, kind):
    """gate+up, and down on rows of its own (as wide as the first multiple of 64 from inter on)."""
    import torch

    print("bf16 experts", t, topk, inter, hidden, counts, kind, flush=True)
    E, P, g = len(counts), t * topk, _gen(inter)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    offsets, live = torch.from_numpy(off).cuda(), int(off[-1])
    pairs = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    token, wide = (pairs // topk).long(), (inter + 63) // 64 * 64
    wm, xm = _middles(kind, 119)
    if kind == "small weights":
        xm = 239  # the gate's sums of order 1
    gate, up, x = Mat(wq, g, E, inter, hidden, wm), Mat(wq, g, E, inter, hidden, wm), Mat(wq, g, 1, t, hidden, xm)
    down, h = Mat(wq, g, E, hidden, wide, wm), Mat(wq, g, 1, P, wide, xm)
    if kind == "nan":
        for e in range(E):
            for r in EDGES:
                (gate if (r + e) % 2 else up).nan(e, r, 0 if r % 2 else -1)
                down.nan(e, r, -1 if r % 2 else 0)
            down.nan(e, hidden - 1, -1)
    xv, hv = x.values(), h.values()
    hg = _out(torch, P, inter, "bf16")
    wq.wq_moe_gate_up(xv.to(torch.bfloat16), offsets, pairs, topk, gate.packed(), up.packed(), h=hg)
    assert bool((hg[live:] == 9.0).all()), "rows behind the last expert's were written"
    d = _out(torch, P, hidden, "f32")
    wq.wq_moe_down(hv.to(torch.bfloat16), t, topk, offsets, pairs, down.packed(), d=d)
    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if counts[e] == 0:
            continue
        xe = xv[token[r]]
        ref, bound = _gate_up_bound(*_product(xe, gate.values(e)), *_product(xe, up.values(e)), hidden)
        _within(hg[r], ref, bound, f"gate+up of expert {e} {kind}")
        ref, mag = _product(hv[r], down.values(e))
        _within(d[pairs[r].long()], ref, _sum_bound(ref, mag, wide, "f32"), f"down of expert {e} {kind}")
    assert bool((d[pairs[live:].long()] == 9.0).all()), "a dropped pair's row was written"
