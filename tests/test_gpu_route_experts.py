"""The routing sort over more pairs than its small kernel takes, for numbers of experts that do not
divide the workgroup's threads: every pair is placed."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("chunked", [True, False])
@pytest.mark.parametrize("t,topk,E", [(1025, 4, 7), (400, 3, 3), (2000, 6, 60), (700, 8, 160), (3000, 8, 384), (1000, 2, 500)])
def test_route_every_pair_for_any_number_of_experts(t, topk, E, chunked):
    import torch

    import weight_only_bit_amd as wq

    print("route", t, topk, E, chunked, flush=True)
    ids = np.random.default_rng(E).integers(0, E, (t, topk)).astype(np.int32)
    ids[t // 2, 0] = -1  # a dropped pair
    offsets, pairs = wq.wq_moe_route(torch.from_numpy(ids).cuda(), E, chunked=chunked)
    flat = ids.reshape(-1)
    order = np.argsort(np.where(flat < 0, E, flat), kind="stable")[: flat.size - 1]
    counts = np.bincount(flat[flat >= 0], minlength=E)
    assert np.array_equal(offsets.cpu().numpy(), np.concatenate([[0], np.cumsum(counts)]))
    assert np.array_equal(pairs.cpu().numpy()[: order.size], order)
