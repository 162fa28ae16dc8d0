"""The accuracy of btq_kv_attention over long contexts, apart from its own formula: the
error of whole rows relative to their length, against 64 bits.

A weight p*s' is rounded to bf16, off by at most 2^-8 of itself, so by 2^-8/sqrt(3) in
the mean square if all had the largest step. Over many rows, whose roundings do not
depend on each other, the error of sum p*v/l is then at most
    (2^-8/sqrt(3)) * sqrt(sum (p*v)^2)/l
in the mean square, whatever the number of keys. 5% is for the scatter of 4096 values or
more (1/sqrt(2*4096) is 1%) and the rounding of scores.

Queries of zeros have weights that are exact (p = 1 and s' holds 8 bits). What is left is
the rounding of sums: a value enters as 128 + code, up to 143, and the 128 + z goes off
them behind every 1024 keys. A step of 32 keys is off by at most 2^-24 of a sum that grows
to 143*1024*mean(s'), 2^-24/sqrt(3) in the mean square, which over the window's 32 steps is
    143*1024*s'*(2^-24/sqrt(3))*sqrt(32/3) = 0.0165*s',   0.024*s' for both sums,
and sqrt(L/1024) of that over L keys. The values here, (code - 7 or 8)*s', have 4.6*s' in the
mean square and a sum of 4.6*s'*sqrt(L), so this is 1.6e-4 of the row. 2^-11, three times as
much, is an eighth of a bf16 rounding's most.

lse: a lane adds L/4 weights one by one, 2^-24/sqrt(3) of a growing sum each, 2^-24*sqrt(L/4)/3
in the mean square; the largest of 128 rows is taken as 12 times that at most."""
import numpy as np
import pytest
import torch

import bit_tensor_activation_amd as B
from helpers import say
from kv_helpers import BF16, DEV, block_bytes, host, unpack

PAGE = 1024


def shared_cache(length, Hk, D, seed):
    """A cache of one sequence's pages, of random codes, and its table row."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    pages = -(-length // PAGE)
    shape = (1, pages, Hk, PAGE // 32, block_bytes(D))
    cache = torch.randint(0, 256, shape, generator=g, dtype=torch.uint8, device=DEV)
    words = cache[..., 32 * D:].view(torch.int32)
    bits = torch.randint(0x3e80, 0x3f00, words.shape, generator=g, dtype=torch.int32, device=DEV)
    z = torch.randint(7, 9, words.shape, generator=g, dtype=torch.int32, device=DEV)
    words.copy_(bits << 16 | 0x4300 | z)
    return cache, torch.randperm(pages, generator=g, device=DEV).int()


# sequences (all of the same pages), rows each, features, keys; which kernel it is
CASES = [(1, 1024, 64, 131072, "columns, 32 a wave"), (1, 512, 160, 32768, "columns, 16 a wave"),
         (64, 1, 64, 131072, "whole groups of 8"), (64, 1, 160, 65536, "whole groups of 16"),
         (32, 1, 64, 131072, "equal shares")]


@pytest.mark.gpu
@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("n", range(len(CASES)))
def test_error_does_not_grow_with_the_context(n, zero):
    seqs, new, D, length, what = CASES[n]
    say(f"case: kv attention over {length} keys, D={D}, {what}, zero queries {zero}")
    Hk, rows = 64, min(seqs * new, 64)
    cache, order = shared_cache(length, Hk, D, n)
    T = seqs * new
    g = torch.Generator(device=DEV).manual_seed(n)
    # scores of some 0.5 in the mean square
    q = 0.3 * torch.randn((1, T, Hk, D), generator=g, device=DEV).to(BF16) * (0 if zero else 1)
    starts = torch.arange(0, T + 1, new, dtype=torch.int32, device=DEV)
    lengths = torch.full((seqs,), length, dtype=torch.int32, device=DEV)
    tb = order.repeat(seqs, 1)
    lse = torch.empty((1, T, Hk), device=DEV)
    out = B.btq_kv_attention(q, starts, lengths, tb, cache, out_dtype=torch.float32, lse=lse)
    out, lse, q, order = host(out).reshape(T, Hk, D), host(lse)[0], host(q)[0], order.cpu().numpy()
    off, most = [], []
    for h in (0, Hk - 1):
        k, v = (x[0, order, 0].reshape(-1, D)[:length] for x in unpack(cache[:, :, h:h + 1].cpu().numpy(), D))
        at = length - new + np.arange(T - rows, T) % new      # the last rows' places
        t = q[T - rows:, h] @ k.T * D ** -0.5
        t[np.arange(length) > at[:, None]] = -np.inf
        m = t.max(-1, keepdims=True)
        p = np.exp(t - m)
        total = p.sum(-1, keepdims=True)
        off.append(out[T - rows:, h] - p @ v / total)
        most.append(np.sqrt(p ** 2 @ v ** 2) / total)
        exact = m[:, 0] + np.log(total[:, 0])
        assert np.abs(lse[T - rows:, h] - exact).max() <= 2.0 ** -22 * (np.sqrt(length / 4) + np.abs(exact).max())
    off, most = (np.sqrt(np.mean(np.square(x))) for x in (off, most))
    say(f"  error {off / most:.2e} of a row")
    assert off <= (2.0 ** -11 if zero else 1.05 * 2.0 ** -8 / 3 ** 0.5) * most
