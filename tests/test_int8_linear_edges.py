"""The 8-bit linear layer at the limits of its sizes."""
import pytest
import torch

from bit_tensor_activation_amd import _lib


# ---- CPU: all return before any HIP call ---------------------------------------

A = 0x10000


@pytest.mark.parametrize("P,T,K", [(1, 1 << 62, 1), (1, (1 << 60) + 1, 1), (1 << 15, 1 << 46, 1),
                                   (1, 1 << 58, 16), (3, (1 << 58) // 3, 15)])
def test_workspace_size_that_overflows_is_refused(P, T, K):
    # x is inside 2^62 elements; the workspace's padded rows of codes and their
    # scales are not, and P*T*(K rounded up to 16 + 4) wraps to a small number or 0
    lib = _lib.load()
    assert P * T * K <= 1 << 62 < P * T * ((K + 15) // 16 * 16 + 4)
    assert lib.btq_int8_linear_workspace_bytes(P, T, K) == 0
    st = lib.btq_int8_linear(A, 1, 0, 0, A, A, None, P, T, 1, K, A, 1, A, (1 << 63) - 1, None)
    assert st == _lib.BTQ_ERR_SHAPE


def test_largest_workspace():
    lib = _lib.load()
    assert lib.btq_int8_linear_workspace_bytes(1, 1 << 57, 16) == 20 << 57
    assert lib.btq_int8_linear_workspace_bytes(1, 1 << 40, 131071) == 131076 << 40
