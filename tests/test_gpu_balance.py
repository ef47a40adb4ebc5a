"""The routing's balance loss, the experts' counts and the logits' gradient on the GPU against the definition
in 64 bits (i8_testutil)."""
import numpy as np
import pytest

import i8_testutil as i8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def wq():
    import torch

    import weight_only_bit_amd as wq

    assert torch.cuda.is_available(), "GPU tests need a GPU"
    wq.lib()
    return wq


def _inputs(t, topk, E, dtype, seed=0):
    import torch

    rng = np.random.default_rng(seed)
    z = torch.from_numpy(rng.standard_normal((t, E)) * 3).to(torch.float32 if dtype == "f32" else torch.bfloat16)
    ids = rng.integers(0, E, (t, topk)).astype(np.int32)
    return z, ids


def _check(wq, z, ids, dtype, coefficient=0.01, d_loss=None, counts=None, what=""):
    """Loss, counts and gradient against the bounds; returns them."""
    import torch

    zc, ic = z.cuda(), torch.from_numpy(ids).cuda()
    dl = None if d_loss is None else torch.tensor(d_loss, device="cuda")
    loss, got = wq.wq_moe_balance_loss(zc, ic, coefficient)
    use = got if counts is None else torch.from_numpy(counts.astype(np.int32)).cuda()
    d = wq.wq_moe_balance_loss_grad(zc, ic, use, coefficient, dl)
    ref, bound, mine, rd, bd = i8.balance_bounds(z.double().numpy(), ids, coefficient, dtype,
                                                 1.0 if d_loss is None else float(np.float32(d_loss)), counts)
    assert loss.shape == () and loss.dtype == torch.float32
    assert np.array_equal(got.cpu().numpy(), mine), what
    i8.assert_within(loss.item(), ref, bound + 2.0 ** -140, what + " loss")
    i8.assert_within(i8.to_host(d), rd, bd, what + " d_logits")
    return loss, got, d


# groups of 1 to 64 lanes, several logits a lane, numbers that no group has, one workgroup and many
SIZES = [(1, 1, 1), (1, 2, 2), (7, 1, 3), (32, 2, 4), (300, 2, 8), (1000, 3, 17), (5000, 4, 32), (64, 8, 60),
         (4096, 8, 64), (33, 8, 65), (700, 8, 128), (100, 6, 160), (3000, 8, 256), (1, 8, 257), (1200, 8, 512), (20, 70, 5)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("t,topk,E", SIZES)
def test_loss_and_gradient(wq, dtype, t, topk, E):
    print("balance", dtype, t, topk, E, flush=True)
    z, ids = _inputs(t, topk, E, dtype, t)
    _check(wq, z, ids, dtype, what="plain")
    # ids outside the experts on either side, and tokens without any
    rng = np.random.default_rng(t + 1)
    ids[rng.random(ids.shape) < 0.2] = -1
    ids[rng.random(ids.shape) < 0.1] = E
    ids[rng.random(ids.shape) < 0.02] = 2**31 - 1
    ids[t - t // 3:] = -1
    _check(wq, z, ids, dtype, 1.5, -0.3, what="padded")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E", [4, 64, 160])
def test_padding_holds_anything(wq, dtype, E):
    """NaN and infinities among padding's logits reach nothing; its gradient is zero."""
    import torch

    z, ids = _inputs(50, 2, E, dtype, 3)
    ids[10:20] = -1
    ids[45:] = E
    base = _check(wq, z, ids, dtype)
    z[10:15] = float("nan")
    z[15:20] = float("inf")
    z[45:] = -float("inf")
    zc, ic = z.cuda(), torch.from_numpy(ids).cuda()
    loss, counts = wq.wq_moe_balance_loss(zc, ic, 0.01)
    d = wq.wq_moe_balance_loss_grad(zc, ic, counts, 0.01)
    assert torch.equal(loss, base[0]) and torch.equal(counts, base[1]) and torch.equal(d, base[2])
    assert (d[10:20] == 0).all() and (d[45:] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_experts_and_extremes(wq, dtype):
    """Logits of -inf have no probability and no gradient, also a whole row; the type's lowest value is a
    number; far-apart logits leave one probability; a NaN of a token makes the loss NaN."""
    import torch

    for E in (8, 64, 100):
        z, ids = _inputs(40, 2, E, dtype, 5)
        z[:10, 1] = -float("inf")
        z[10] = -float("inf")
        z[11] = torch.finfo(z.dtype).min
        z[12, :] = torch.finfo(z.dtype).min
        z[12, 3] = 0
        z[13] = torch.finfo(z.dtype).max
        z[14, 0], z[14, 1:] = 1e4, -1e4
        zc, ic = z.cuda(), torch.from_numpy(ids).cuda()
        loss, counts = wq.wq_moe_balance_loss(zc, ic)
        d = wq.wq_moe_balance_loss_grad(zc, ic, counts)
        ref, mine, rd, p, _ = i8.balance(z.double().numpy(), ids, 1.0)
        assert np.array_equal(counts.cpu().numpy(), mine)
        # differences of these rows are exact or leave e^x = 0, but for the ordinary rows' (span 30)
        rel = 64 * 2.0 ** -23
        assert abs(loss.item() - ref) <= abs(ref) * (rel + 350 * i8.U)
        share = E * mine[:E] / mine[:E].sum()
        mags = p * (share + (p * share).sum(1, keepdims=True)) / mine[E]
        i8.assert_within(i8.to_host(d), rd, 4 * rel * mags + i8.HALF[dtype] * np.abs(rd) + 2.0 ** -133, "d")
        assert (d[:10, 1] == 0).all() and (d[10] == 0).all()
        z[20, 2] = float("nan")
        loss, counts = wq.wq_moe_balance_loss(z.cuda(), ic)
        d = wq.wq_moe_balance_loss_grad(z.cuda(), ic, counts)
        assert loss.isnan() and d[20].isnan().all() and d[21:].isfinite().all() and d[:20].isfinite().all()


def test_nothing_to_count(wq):
    import torch

    for t in (0, 5, 3000):
        z = torch.randn(t, 64, device="cuda")
        ids = torch.full((t, 4), -1, dtype=torch.int32, device="cuda")
        loss, counts = wq.wq_moe_balance_loss(z, ids)
        assert loss.item() == 0 and (counts == 0).all()
        d = wq.wq_moe_balance_loss_grad(z, ids, counts)
        assert d.shape == (t, 64) and (d == 0).all()


def test_counts_of_several_calls(wq):
    """Shards of a batch: the gradients with the summed counts are those of the whole batch, whose loss has
    the shares of all tokens."""
    import torch

    z, ids = _inputs(999, 4, 60, "f32", 11)
    zc, ic = z.cuda(), torch.from_numpy(ids).cuda()
    loss, counts = wq.wq_moe_balance_loss(zc, ic, 0.5)
    whole = wq.wq_moe_balance_loss_grad(zc, ic, counts, 0.5)
    parts = [slice(0, 400), slice(400, 401), slice(401, 999)]
    total = sum(wq.wq_moe_balance_loss(zc[s], ic[s])[1] for s in parts)
    assert torch.equal(total, counts)
    for s in parts:
        assert torch.equal(wq.wq_moe_balance_loss_grad(zc[s], ic[s], total, 0.5), whole[s])
    _check(wq, z[:400], ids[:400], "f32", 0.5, 2.0, counts.cpu().numpy().astype(np.int64))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("E", [1, 4, 8, 60, 512])
def test_experts_used_alike(wq, dtype, E):
    """Equal counts have no gradient; of counts a millionth apart it keeps its digits: each value's error is the
    probabilities' (spans below 24 and sums of up to 512: under 64 * 2^-23) relative to what it is made of, the shares'
    distances from the mean, not the shares."""
    import torch

    z, ids = _inputs(200, 2, E, dtype, 21)
    zc, ic = z.cuda(), torch.from_numpy(ids).cuda()
    pairs = np.full(E, 10**6, dtype=np.int64)
    counts = np.append(pairs, 200)
    d = wq.wq_moe_balance_loss_grad(zc, ic, torch.from_numpy(counts.astype(np.int32)).cuda(), 0.5)
    assert (d == 0).all()
    pairs += np.arange(E) % 3
    counts = np.append(pairs, 200)
    d = wq.wq_moe_balance_loss_grad(zc, ic, torch.from_numpy(counts.astype(np.int32)).cuda(), 0.5)
    x = z.double().numpy()
    p = np.exp(x - x.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    over = (E * pairs - pairs.sum()) / pairs.sum()  # whole numbers, one rounding
    rd = 0.5 / 200 * p * (over - (p * over).sum(1, keepdims=True))
    mags = 0.5 / 200 * p * (np.abs(over) + (p * np.abs(over)).sum(1, keepdims=True))
    i8.assert_within(i8.to_host(d), rd, 4 * 64 * 2.0 ** -23 * mags + i8.HALF[dtype] * np.abs(rd) + 2.0 ** -133, "d")


def test_gradient_against_differences(wq):
    rng = np.random.default_rng(2)
    z, ids = _inputs(60, 3, 20, "f32", 12)
    ids[50:] = -1
    _, _, d = _check(wq, z, ids, "f32", 1.0)
    f = lambda v: i8.balance(v, ids, 1.0)[0]
    h = 1e-5
    for _ in range(4):
        u = rng.standard_normal(z.shape)
        diff = (f(z.double().numpy() + h * u) - f(z.double().numpy() - h * u)) / (2 * h)
        assert abs(diff - (i8.to_host(d) * u).sum()) < 1e-5 * np.abs(i8.to_host(d) * u).sum()


def test_large_batches_repeat_bit_for_bit(wq):
    """Many workgroups: the same bits every time, counts and the loss's value against torch in fp64."""
    import torch

    for t, E in ((65536, 256), (200003, 64), (1000003, 8)):
        z = torch.randn(t, E, device="cuda")
        ids = torch.randint(0, E, (t, 2), device="cuda", dtype=torch.int32)
        loss, counts = wq.wq_moe_balance_loss(z, ids)
        d = wq.wq_moe_balance_loss_grad(z, ids, counts)
        want = torch.bincount(ids.reshape(-1).long(), minlength=E)
        assert torch.equal(counts[:E].long(), want) and counts[E].item() == t
        p = torch.softmax(z.double(), 1).mean(0)
        ref = (E * want / want.sum() * p).sum().item()
        assert abs(loss.item() - ref) < 1e-5 * ref
        for _ in range(2):
            again = wq.wq_moe_balance_loss(z, ids)
            assert torch.equal(again[0], loss) and torch.equal(again[1], counts)
            assert torch.equal(wq.wq_moe_balance_loss_grad(z, ids, counts), d)
