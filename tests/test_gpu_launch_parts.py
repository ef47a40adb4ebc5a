"""Sizes whose grids hold more threads than one launch may: MXFP4 quantisation and dequantisation, the
permutation, the way back and its gradient.  All values are small integers (or zero), so every result
is exact."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wq():
    import torch

    import weight_only_bit_amd as wq

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    wq.lib()
    yield wq
    torch.cuda.empty_cache()


def _room(gib):
    import torch

    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of free device memory")


def test_rows_of_one_value(wq):
    import torch

    _room(12)
    t = 2**29 + 5  # 32 tokens a workgroup
    print("permute", t, flush=True)
    x = torch.arange(t, dtype=torch.int32, device="cuda").remainder_(251).to(torch.bfloat16).view(t, 1)
    positions = torch.arange(t - 1, -1, -1, dtype=torch.int32, device="cuda").view(t, 1)
    rows = wq.wq_moe_permute(x, positions)
    assert torch.equal(rows[:1000], x[-1000:].flip(0)) and torch.equal(rows[-1000:], x[:1000].flip(0))
    y = wq.wq_moe_unpermute(rows, positions)
    assert torch.equal(x, y)


def test_gradient_of_many_pairs(wq):
    import torch

    _room(12)
    t, topk, hidden = 2**24 + 3, 4, 8  # 4 pairs a workgroup
    P = t * topk
    print("gradient", P, flush=True)
    dy = torch.randint(-8, 9, (t, hidden), dtype=torch.int8, device="cuda").to(torch.bfloat16)
    rows = torch.randint(-8, 9, (P, hidden), dtype=torch.int8, device="cuda").to(torch.bfloat16)
    positions = torch.arange(P - 1, -1, -1, dtype=torch.int32, device="cuda").view(t, topk)
    d_rows, d_w = wq.wq_moe_unpermute_grad(dy, rows, positions)
    for a, b in ((0, 5000), (t - 5000, t)):
        own = rows[P - b * topk:P - a * topk].flip(0).view(b - a, topk, hidden).float()
        g = dy[a:b].float().unsqueeze(1)
        assert torch.equal(d_w[a:b], (own * g).sum(-1))
        got = d_rows[P - b * topk:P - a * topk].flip(0).view(b - a, topk, hidden).float()
        assert torch.equal(got, g.expand_as(got))


def test_mxfp4_of_many_values(wq):
    import torch

    _room(100)
    k = 8192
    n = 2**32 * 8 // k + 40  # 8 values a thread
    print("quantize", n, k, flush=True)
    x = torch.zeros((n, k), dtype=torch.bfloat16, device="cuda")
    tail = torch.randint(-6, 7, (64, k), dtype=torch.int8, device="cuda").to(torch.bfloat16)
    tail[tail.abs() == 5] = 6
    tail[:, ::32] = 6  # every block's scale is 1
    x[:64] = tail
    x[-64:] = tail
    w = wq.wq_quantize_mx(x)
    codes, scales = w.codes[0], w.qscale[0]
    del x
    torch.cuda.empty_cache()
    assert bool((scales[-64:] == 127).all()) and bool((scales[64:-64] == 0).all())
    assert torch.equal(codes[-64:], codes[:64])
    out = wq.wq_dequantize(w).view(n, k).view(torch.bfloat16)
    assert torch.equal(out[:64], tail) and torch.equal(out[-64:], tail)
    assert not bool(out[64:2000].any()) and not bool(out[-2000:-64].any())
