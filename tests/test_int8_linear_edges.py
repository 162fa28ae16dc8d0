"""The 8-bit linear layer at the limits of its sizes."""
import pytest
import torch

import bit_tensor_activation_amd as B
from bit_tensor_activation_amd import _lib
from helpers import say

DEV = torch.device("cuda:0")


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


# ---- GPU -----------------------------------------------------------------------

@pytest.mark.gpu
def test_many_tiles_take_the_tiled_kernel():
    # 2^23 tiles of 32 x 32 (a few less on the other side), and a 64th of that of
    # 256 x 256, which are what runs: the kernel may not change between them.
    # The general kernel takes 3 times as long or more at this K; 1.5 tells
    # them apart, and the products differ by 0.1%.
    P, T, K, N = 8, 32768, 1024, 32768
    say(f"case: int8_matmul P={P} T={T} N={N} K={K}")
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    a = torch.randint(-128, 128, (P, T, K), device=DEV, generator=g, dtype=torch.int8)
    w = torch.randint(-128, 128, (P, N, K), device=DEV, generator=g, dtype=torch.int8)
    sa = torch.rand((P, T), device=DEV, generator=g)
    sw = torch.rand((P, N), device=DEV, generator=g)
    out = torch.empty(P * T * N, dtype=torch.bfloat16, device=DEV)

    def product(n):
        wn, swn = w[:, :n].contiguous(), sw[:, :n].contiguous()
        y = out[:P * T * n].view(P, T, n)
        us = []
        for _ in range(3):
            b, e = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            b.record()
            B.btq_int8_matmul(a, sa, wn, swn, y=y)
            e.record()
            torch.cuda.synchronize()
            us.append(b.elapsed_time(e) * 1e3)
        say(f"  N={n}: {min(us):.0f} us")
        return y, min(us)
    _, below = product(N - 32)
    y, us = product(N)
    rows = torch.tensor([0, 1, 31, 32, 255, 256, T // 2, T - 257, T - 2, T - 1], device=DEV)
    for p in range(P):
        acc = a[p, rows].double() @ w[p].double().t().contiguous()
        want = (acc.float() * sa[p, rows][:, None] * sw[p][None, :]).to(torch.bfloat16)
        assert torch.equal(y[p, rows], want), p
    assert us < 1.5 * below
