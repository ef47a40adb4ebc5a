"""Rows that no pair has, in arrays that the dispatch allocates itself: dropped pairs leave some, and they
are zeros in wq_moe_permute's rows and in wq_moe_unpermute_grad's d_rows, whatever the memory held
before.  All t*topk rows are compared, and all of it is copies and zeros, so every comparison is exact."""
import ctypes

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

TYPES = {"bf16": ("bfloat16", 0), "f32": ("float32", 1)}
# one pair to 40000 (more than one of the clearing workgroups' 128 rows), counts that no 4 divides, rows
# shorter than 16 bytes, rows that end inside a piece, short rows of many pairs (filled beforehand)
SIZES = [(1, 1, 1), (7, 3, 7), (40, 8, 64), (33, 9, 1027), (300, 4, 2049), (5000, 8, 300), (5000, 8, 520), (9000, 4, 5)]


@pytest.fixture(scope="module")
def wq():
    import torch

    import weight_only_bit_amd as wq

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    wq.lib()
    return wq


def _positions(rng, t, topk, kind):
    """Expert order ("tail": kept pairs take the first rows) or rows with holes anywhere."""
    P = t * topk
    pos = rng.permutation(P).astype(np.int32)
    if kind == "none":
        return pos.reshape(t, topk)
    drop = np.ones(P, bool) if kind == "all" else rng.random(P) < 0.3
    if kind == "tail":
        kept = int((~drop).sum())
        pos = np.empty(P, np.int32)
        pos[~drop] = rng.permutation(kept)
    pos[drop] = -1
    return pos.reshape(t, topk)


def _poison(torch, P, hidden, dt):
    """A block that the allocator gives out next, full of NaN."""
    torch.cuda.synchronize()
    block = torch.full((P, hidden), float("nan"), dtype=dt, device="cuda")
    torch.cuda.synchronize()
    del block


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["tail", "holes", "none", "all"])
@pytest.mark.parametrize("t,topk,hidden", SIZES)
def test_rows_of_no_pair_are_zero(wq, t, topk, hidden, kind, dtype):
    import torch

    print("rows of no pair", t, topk, hidden, kind, dtype, flush=True)
    rng = np.random.default_rng(t + hidden)
    P, (name, ty) = t * topk, TYPES[dtype]
    dt = getattr(torch, name)
    pos = _positions(rng, t, topk, kind)
    x = torch.from_numpy(rng.standard_normal((t, hidden)).astype(np.float32)).to(dt)
    want = torch.zeros((P, hidden), dtype=dt)
    token = torch.arange(P) // topk
    flat = torch.from_numpy(pos.reshape(-1).astype(np.int64))
    want[flat[flat >= 0]] = x[token[flat >= 0]]
    xd, pd, want = x.cuda(), torch.from_numpy(pos).cuda(), want.cuda()
    _poison(torch, P, hidden, dt)
    assert torch.equal(wq.wq_moe_permute(xd, pd), want)
    rows = torch.zeros((P, hidden), dtype=dt, device="cuda")
    _poison(torch, P, hidden, dt)
    assert torch.equal(wq.wq_moe_unpermute_grad(xd, None, pd)[0], want)
    _poison(torch, P, hidden, dt)
    assert torch.equal(wq.wq_moe_unpermute_grad(xd, rows, pd)[0], want)
    # the C calls with a buffer that holds NaN
    L, vp = wq.lib(), ctypes.c_void_p
    for clear in (0x100, 0):
        for grad in (False, True):
            out = torch.full((P, hidden), float("nan"), dtype=dt, device="cuda")
            if grad:
                st = L.wq_moe_unpermute_grad(vp(xd.data_ptr()), ty | clear, None, vp(pd.data_ptr()), None, t, topk, hidden,
                                             vp(out.data_ptr()), None, wq._stream())
            else:
                st = L.wq_moe_permute(vp(xd.data_ptr()), ty | clear, t, topk, hidden, vp(pd.data_ptr()),
                                      vp(out.data_ptr()), wq._stream())
            assert st == 0, L.wq_last_error()
            free = torch.ones(P, dtype=torch.bool)
            free[flat[flat >= 0]] = False
            free = free.cuda()
            if clear:
                assert torch.equal(out, want)
            else:
                assert torch.equal(out[~free], want[~free]) and bool(out[free].isnan().all())


def test_weight_gradient_over_all_rows(wq):
    """d_rows^T rows over every row, as a weight's gradient is taken, with pairs dropped: finite and that
    of the kept pairs."""
    import torch

    rng = np.random.default_rng(3)
    t, topk, hidden = 60, 4, 48
    pos = _positions(rng, t, topk, "tail")
    x, dy = (torch.from_numpy(rng.integers(-4, 5, (t, hidden))).float() for _ in range(2))
    pd = torch.from_numpy(pos).cuda()
    _poison(torch, t * topk, hidden, torch.float32)
    rows = wq.wq_moe_permute(x.cuda(), pd)
    _poison(torch, t * topk, hidden, torch.float32)
    d_rows, _ = wq.wq_moe_unpermute_grad(dy.cuda(), rows, pd)
    kept = torch.from_numpy((pos >= 0).sum(1)).float()
    want = (dy * kept[:, None]).t() @ x  # small integers: exact
    assert torch.equal((d_rows.t().contiguous() @ rows).cpu(), want)


def test_captured_with_drops(wq):
    """The clearing launches in a graph, replayed on other positions."""
    import torch

    rng = np.random.default_rng(5)
    for t, topk, hidden in ((200, 4, 640), (9000, 4, 5)):
        print("captured", t, topk, hidden, flush=True)
        live = torch.from_numpy(_positions(rng, t, topk, "tail")).cuda()
        x = torch.from_numpy(rng.standard_normal((t, hidden))).to(torch.bfloat16).cuda()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            wq.wq_moe_permute(x, live)
            wq.wq_moe_unpermute_grad(x, None, live)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            rows = wq.wq_moe_permute(x, live)
            d_rows = wq.wq_moe_unpermute_grad(x, None, live)[0]
        for kind in ("holes", "tail", "none", "all"):
            pos = torch.from_numpy(_positions(rng, t, topk, kind)).cuda()
            want = torch.zeros_like(rows)
            flat = pos.view(-1).long()
            keep = flat >= 0
            want[flat[keep]] = x[(torch.arange(t * topk, device="cuda") // topk)[keep]]
            live.copy_(pos)
            rows.fill_(float("nan"))
            d_rows.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(rows, want) and torch.equal(d_rows, want), kind


def test_many_pairs(wq):
    """Enough pairs that the clearing workgroups are limited by the rows that one can mark."""
    import torch

    t, topk, hidden = 1_100_000, 4, 256
    P = t * topk
    print("many pairs", P, flush=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    drop = torch.rand(P, generator=g, device="cuda") < 0.3
    pos = torch.full((P,), -1, dtype=torch.int32, device="cuda")
    pos[~drop] = torch.randperm(P, generator=g, device="cuda")[: int((~drop).sum())].to(torch.int32)
    x = torch.randint(1, 100, (t, hidden), generator=g, device="cuda", dtype=torch.int8).to(torch.bfloat16)
    _poison(torch, P, hidden, torch.bfloat16)
    rows = wq.wq_moe_permute(x, pos.view(t, topk))
    free = torch.ones(P, dtype=torch.bool, device="cuda")
    free[pos[~drop].long()] = False
    assert not bool(rows[free].any()) and not bool(rows.isnan().any())
    sums = torch.zeros(P, device="cuda")
    sums[pos[~drop].long()] = x.float().sum(1)[(torch.arange(P, device="cuda") // topk)[~drop]]
    assert torch.equal(rows.float().sum(1), sums)  # whole numbers below 2^24: exact
    del rows
    _poison(torch, P, hidden, torch.bfloat16)
    d_rows = wq.wq_moe_unpermute_grad(x, None, pos.view(t, topk))[0]
    assert torch.equal(d_rows.float().sum(1), sums) and not bool(d_rows[free].any())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_beyond_4_gib(wq, dtype):
    """Permutation, way back and gradients over rows of 8.6 GB, a fifth of the pairs dropped."""
    import torch

    t, topk, hidden = (1 << 16) + 3, 8, 8192 if dtype == "bf16" else 4096
    P, dt = t * topk, getattr(torch, TYPES[dtype][0])
    print("rows beyond 4 GiB", P, hidden, dtype, flush=True)
    g = torch.Generator(device="cuda").manual_seed(2)
    drop = torch.rand(P, generator=g, device="cuda") < 0.2
    kept = int((~drop).sum())
    pos = torch.full((P,), -1, dtype=torch.int32, device="cuda")
    pos[~drop] = torch.randperm(kept, generator=g, device="cuda").to(torch.int32)
    x = torch.randint(-8, 9, (t, hidden), generator=g, device="cuda", dtype=torch.int8).to(dt)
    pos = pos.view(t, topk)
    rows = wq.wq_moe_permute(x, pos)
    owner = torch.full((P,), -1, dtype=torch.int64, device="cuda")  # the token of every row
    owner[pos.view(-1)[~drop].long()] = (torch.arange(P, device="cuda") // topk)[~drop]
    assert not bool(rows[kept:].any())
    for r in (slice(0, 500), slice(kept // 2, kept // 2 + 500), slice(kept - 500, kept)):
        assert torch.equal(rows[r], x[owner[r]])
    # whole numbers: a token's kept rows are copies of it
    n = (pos >= 0).sum(1, keepdim=True).float()
    y = wq.wq_moe_unpermute(rows, pos)
    for s in (slice(0, 300), slice(t - 300, t)):
        assert torch.equal(y[s].float(), x[s].float() * n[s])
    d_rows, d_w = wq.wq_moe_unpermute_grad(x, rows, pos)
    assert not bool(d_rows[kept:].any())
    for r in (slice(0, 500), slice(kept - 500, kept)):
        assert torch.equal(d_rows[r], x[owner[r]])
    for s in (slice(0, 300), slice(t - 300, t)):
        assert torch.equal(d_w[s], (pos[s] >= 0).float() * (x[s].float() ** 2).sum(1, keepdim=True))
