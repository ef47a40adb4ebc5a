"""Every int8 product kernel, the norm's shapes and the balance loss's launches captured and replayed over new inputs, and
on two streams at once."""
import pytest

from i8_cases import DENSE, EXPERTS

pytestmark = pytest.mark.gpu

# the first case of each kernel
ONE_OF_EACH = list({c.kernel: c for c in reversed(DENSE)}.values())
EXPERTS_OF_EACH = list({(c.kernel, c.gate_up): c for c in reversed(EXPERTS)}.values())


@pytest.fixture(scope="module")
def wq():
    import torch

    import weight_only_bit_amd as wq

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    wq.lib()
    return wq


def _codes(*shape):
    import torch

    return torch.randint(-128, 128, shape, dtype=torch.int8, device="cuda")


def _weight(wq, E, n, k):
    import torch

    return wq.PackedWeight(wq.FMT_INT8, n, k, E, 0, codes=_codes(E, n, k),
                           scales=(torch.rand((E, n), device="cuda") * 1e-3).to(torch.bfloat16))


def _all(v):
    """The tensors of a call's result."""
    if isinstance(v, tuple):
        return [t for x in v for t in _all(x)]
    return [v]


def _captured(call, refresh):
    """call() captured once; each replay over refreshed inputs, with eager work between, is what call() gives eagerly."""
    import torch

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _all(call())
    for i in range(3):
        refresh()
        want = [t.clone() for t in _all(call())]
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i


def _two_streams(calls):
    """The calls on two streams at once, several times, give what each gives alone."""
    import torch

    want = [[t.clone() for t in _all(c())] for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[] for _ in calls]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for i, (s, c) in enumerate(zip(streams, calls)):
            with torch.cuda.stream(s):
                got[i].append(_all(c()))
    torch.cuda.synchronize()
    for i in range(len(calls)):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i])), i


@pytest.mark.parametrize("case", ONE_OF_EACH, ids=lambda c: c.kernel)
def test_dense_products(wq, case):
    import torch

    print("dense", case, flush=True)
    w = [_weight(wq, 1, case.n, case.k) for _ in range(2)]
    x = [wq.Int8Rows(_codes(case.m, case.k), torch.rand(case.m, device="cuda")) for _ in range(2)]
    _captured(lambda: wq.wq_gemm_i8(x[0], w[0]), lambda: x[0].codes.copy_(_codes(case.m, case.k)))
    _two_streams([lambda i=i: wq.wq_gemm_i8(x[i], w[i]) for i in range(2)])


@pytest.mark.parametrize("case", EXPERTS_OF_EACH, ids=lambda c: f"{c.kernel}-{'up' if c.gate_up else 'down'}")
def test_experts_products(wq, case):
    import torch

    print("experts", case, flush=True)
    E, pairs = len(case.counts), case.t * case.topk
    ids = torch.full((pairs,), -1, dtype=torch.int32)
    ids[torch.randperm(pairs)[: sum(case.counts)]] = torch.repeat_interleave(torch.arange(E), torch.tensor(case.counts)).int()
    ids = ids.view(case.t, case.topk).cuda()
    rows = case.t if case.gate_up else pairs
    g, u = _weight(wq, E, case.n, case.k), _weight(wq, E, case.n, case.k)
    x = [wq.Int8Rows(_codes(rows, case.k), torch.rand(rows, device="cuda") * 0.01) for _ in range(2)]

    def call(i=0):
        off, order = wq.wq_moe_route(ids, E)
        out = torch.zeros((pairs, case.n), dtype=torch.bfloat16, device="cuda")
        if case.gate_up:
            return wq.wq_moe_gate_up_i8(x[i], off, order, case.topk, g, u, h=out)
        return wq.wq_moe_down_i8(x[i], off, g, d=out)

    def refresh():
        x[0].codes.copy_(_codes(rows, case.k))
        ids.copy_(ids[torch.randperm(case.t, device="cuda")])

    _captured(call, refresh)
    _two_streams([lambda i=i: call(i) for i in range(2)])


# rows of every number of lanes, one workgroup's gradient and many, rows that are read again
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,k", [(1, 64), (300, 100), (300, 1000), (40, 1111), (700, 4099), (33, 8192), (300, 12000), (5, 70003)])
def test_norms(wq, dtype, n, k):
    import torch

    print("norms", dtype, n, k, flush=True)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    v = [[torch.randn((n, k), device="cuda").to(dt) for _ in range(4)] for _ in range(2)]
    w = torch.randn(k, device="cuda").to(dt)

    def call(i=0):
        x, res, dy, ds = v[i]
        y, total = wq.wq_rms_norm(x, w, res)
        return y, total, wq.wq_rms_norm_i8(x, w, res), wq.wq_quantize_i8(x), wq.wq_rms_norm_grad(dy, total, w, ds)

    def refresh():
        for t in v[0]:
            t.copy_(torch.randn((n, k), device="cuda"))

    _captured(call, refresh)
    _two_streams([lambda i=i: call(i) for i in range(2)])


# one workgroup, parts that one launch adds, parts that two add
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,E", [(50, 8), (4096, 64), (9000, 60), (40000, 256)])
def test_balance(wq, dtype, t, E):
    import torch

    print("balance", dtype, t, E, flush=True)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    v = [(torch.randn((t, E), device="cuda").to(dt), torch.randint(-1, E, (t, 2), device="cuda", dtype=torch.int32))
         for _ in range(2)]

    def call(i=0):
        loss, counts = wq.wq_moe_balance_loss(*v[i], 0.01)
        return loss, counts, wq.wq_moe_balance_loss_grad(*v[i], counts, 0.01)

    def refresh():
        v[0][0].copy_(torch.randn((t, E), device="cuda"))
        v[0][1].copy_(torch.randint(-1, E, (t, 2), device="cuda", dtype=torch.int32))

    _captured(call, refresh)
    _two_streams([lambda i=i: call(i) for i in range(2)])


def test_each_kernel_is_there():
    from i8_cases import KERNELS

    assert {c.kernel for c in ONE_OF_EACH} == set(KERNELS)
    assert len(EXPERTS_OF_EACH) == 8
