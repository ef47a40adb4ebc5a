"""Digits of the balance loss's probabilities, and padding beside what is not finite, on the GPU against the
definition in 64 bits."""
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


@pytest.mark.parametrize("E", [3, 9, 65, 301])
def test_probabilities_far_from_the_largest(wq, E):
    """Logits of 0 and of -20 to -70: the differences from the maximum are exact, so a probability's error holds no
    multiple of them.  Counts under which expert 0 has the mean share, so that the gradients of the others are their
    probability times their share's distance: off by the exponential (3 roundings), its sum (a chain of 16 + 5) and the
    sum's reciprocal, the slope, the factor, the share (3), its distance and two products."""
    import torch

    rng = np.random.default_rng(E)
    t = 300
    z = -rng.uniform(20, 70, (t, E)).astype(np.float32)
    z[:, 0] = 0
    ids = rng.integers(0, E, (t, 2)).astype(np.int32)
    pairs = np.full(E, 10000)
    pairs[1::2] += 7000
    pairs[2::2] -= 7000
    counts = np.append(pairs, t)
    d = wq.wq_moe_balance_loss_grad(torch.from_numpy(z).cuda(), torch.from_numpy(ids).cuda(),
                                    torch.from_numpy(counts.astype(np.int32)).cuda())
    p = np.exp(z.astype(np.float64))
    p /= p.sum(1, keepdims=True)
    over = (E * pairs - pairs.sum()) / pairs.sum()
    assert over[0] == 0
    ref = p * (over - (p * over).sum(1, keepdims=True)) / t
    mags = p * (np.abs(over) + (p * np.abs(over)).sum(1, keepdims=True)) / t
    assert mags[:, 1:].min() > 2.0 ** -110
    i8.assert_within(i8.to_host(d), ref, (3 + 21 + 1 + 1 + 1 + 3 + 1 + 2) * i8.U * mags, "d_logits")


def test_probabilities_beside_many_small_ones(wq):
    """One logit of 0 and 14 whose exponentials are a part of 2^-24, too small each to change a sum of one: a chain of
    16 additions loses up to 15 of them, sums of four lose 4 + 2 halves of a step.  Sizes that are powers of two make
    slope and shares exact, so that what is left are the exponential (3), its sum (6), the reciprocal, two products and the
    share's distance."""
    import torch

    E, t = 16, 256
    rng = np.random.default_rng(4)
    z = np.zeros((t, E), np.float32)
    z[:, 1:] = np.log(np.linspace(0.6, 0.99, t))[:, None] - 24 * np.log(2)
    z[:, 15] = -rng.uniform(20, 70, t)
    ids = rng.integers(0, E, (t, 2)).astype(np.int32)
    pairs = np.full(E, 1 << 14)
    pairs[1] -= 1 << 13
    pairs[15] += 1 << 13
    counts = np.append(pairs, t)
    d = wq.wq_moe_balance_loss_grad(torch.from_numpy(z).cuda(), torch.from_numpy(ids).cuda(),
                                    torch.from_numpy(counts.astype(np.int32)).cuda())
    p = np.exp(z.astype(np.float64))
    p /= p.sum(1, keepdims=True)
    over = (E * pairs - pairs.sum()) / pairs.sum()
    ref = p * (over - (p * over).sum(1, keepdims=True)) / t
    mags = p * (np.abs(over) + (p * np.abs(over)).sum(1, keepdims=True)) / t
    some = [1, 15]
    i8.assert_within(i8.to_host(d)[:, some], ref[:, some], (3 + 6 + 1 + 2 + 1) * i8.U * mags[:, some], "d_logits")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d_loss", [float("inf"), float("nan")])
def test_padding_beside_a_loss_that_is_not_finite(wq, dtype, d_loss):
    """Padding's gradient is zero whatever reaches the loss; the tokens' is not finite."""
    import torch

    for E in (3, 8, 64, 300):
        z = torch.randn(40, E, device="cuda").to(torch.float32 if dtype == "f32" else torch.bfloat16)
        ids = torch.randint(0, E, (40, 2), device="cuda", dtype=torch.int32)
        ids[:, 0] = 0  # loaded unevenly: no gradient is zero
        ids[30:] = -1
        _, counts = wq.wq_moe_balance_loss(z, ids)
        d = wq.wq_moe_balance_loss_grad(z, ids, counts, d_loss=torch.tensor(d_loss, device="cuda"))
        assert (d[30:] == 0).all() and not d[:30].isfinite().any()
