"""The token dispatch refuses outputs that share memory with rows or tokens (CPU: nothing is launched).
4 tokens x 2 of 64 values; bf16 rows are 1024 bytes, fp32 rows 2048."""
import pytest

A = 0x10000


@pytest.mark.parametrize("ty,size", [(0, 2), (1, 4)])
def test_overlaps_are_refused(ty, size):
    import weight_only_bit_amd as wq

    L = wq.lib()
    t, k, h = 4, 2, 64
    tokens, rows = t * h * size, t * k * h * size
    pos, far = 0x900000, 0x800000
    for other in (A, A + tokens - 16, A - rows + 16):
        assert L.wq_moe_permute(A, ty, t, k, h, pos, other, None) == -1
        assert "overlap" in L.wq_last_error().decode()
    for other in (A, A + rows - 16, A - tokens + 16):
        assert L.wq_moe_unpermute(A, ty, pos, None, t, k, h, other, None) == -1
    for other in (A, A + tokens - 16, A - rows + 16):
        assert L.wq_moe_unpermute_grad(A, ty, far, pos, None, t, k, h, other, far + rows, None) == -1
    for other in (A, A + rows - 16, A - rows + 16):
        assert L.wq_moe_unpermute_grad(far, ty, A, pos, None, t, k, h, other, None, None) == -1
        assert "overlaps" in L.wq_last_error().decode()
