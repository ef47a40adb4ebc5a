"""The dispatch's WQ_CLEAR_ROWS, added to the element type: taken by the two calls that write rows, refused
by the others and beside a type that is none (CPU: nothing is launched)."""
import ctypes

import pytest

P = [ctypes.c_void_p(0x100000 * (i + 1)) for i in range(6)]


@pytest.fixture(scope="module")
def L():
    import os

    import weight_only_bit_amd as wq

    if not os.path.exists(wq.LIB_PATH):
        from weight_only_bit_amd import build

        build.build()
    return wq.lib()


@pytest.mark.parametrize("ty", [0, 1])
def test_flag_is_taken(L, ty):
    t = 0x100 | ty
    assert L.wq_moe_permute(None, t, 0, 2, 64, None, None, None) == 0
    assert L.wq_moe_permute(P[0], t, 4, 2, 64, P[1], None, None) == -1
    assert L.wq_moe_permute(P[0], t, 4, 2, 64, P[1], P[0], None) == -1  # overlap, with the type's size
    assert L.wq_moe_unpermute_grad(None, t, None, None, None, 0, 2, 64, None, None, None) == 0
    assert L.wq_moe_unpermute_grad(P[0], t, None, P[1], None, 4, 2, 64, None, None, None) == 0  # nothing asked for
    assert L.wq_moe_unpermute_grad(None, t, None, P[1], None, 4, 2, 64, P[2], None, None) == -1


def test_flag_is_refused_elsewhere(L):
    assert L.wq_moe_permute(P[0], 0x102, 4, 2, 64, P[1], P[2], None) == -2
    assert L.wq_moe_permute(P[0], 0x200, 4, 2, 64, P[1], P[2], None) == -2
    assert L.wq_moe_permute(P[0], -1, 4, 2, 64, P[1], P[2], None) == -2
    assert L.wq_moe_unpermute_grad(P[0], 0x107, None, P[1], None, 4, 2, 64, P[2], None, None) == -2
    assert L.wq_moe_unpermute(P[0], 0x100, P[1], None, 4, 2, 64, P[2], None) == -2
    assert L.wq_quantize_mx(P[0], 0x101, 4, 64, P[1], P[2], None) == -2
