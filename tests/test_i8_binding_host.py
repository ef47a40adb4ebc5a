"""CPU tests of what the binding says of arguments that are no tensors."""
import numpy as np
import pytest

from test_abi import wq  # noqa: F401  (fixture)


def test_ids_that_are_no_tensor(wq):  # noqa: F811
    import torch

    z, ids = torch.zeros((2, 64)), np.zeros((2, 2), np.int32)
    for call in (lambda: wq.wq_moe_balance_loss(z, ids), lambda: wq.wq_moe_balance_loss_grad(z, ids, torch.zeros(65))):
        with pytest.raises(TypeError, match="topk_ids: expected a torch tensor"):
            call()
