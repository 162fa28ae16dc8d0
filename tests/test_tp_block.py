"""The whole tensor-parallel boundary (tp_block.py): 8-bit linear layer, sender,
receiver, block norm and the next product, run together.

What the error of y has to be. Two parts add up in y: the 8-bit codes of the
linear layer, at most 2% of it (normal rows of 512: the largest value is below
4.4 sigma, so sqrt(2)*4.4/127/sqrt(12) = 1.4%), and the codec's int4 rounding,
uniform over a step of scale[p,h] for each shard and int4 feature: a variance of
sum_p scale^2/12, known from the calibrated scales. Values beyond the calibrated
range are clamped and add to it; the check allows 1.5 times the predicted root.
"""
import pytest
import torch

import tp_block as X
from helpers import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P,T,H,K,N,k", [(8, 64, 1024, 512, 256, 32), (4, 1, 512, 512, 128, 16),
                                         (2, 300, 1016, 640, 136, 24), (8, 256, 2048, 512, 512, 0)])
def test_step_against_unquantized_values(P, T, H, K, N, k):
    say(f"case: tensor-parallel block P={P} T={T} H={H} K={K} N={N} k={k}")
    s = X.prepare(P, T, H, K, N, k)
    y, residual, z = X.step(s)
    want_y, want_r, want_z = X.exact(s)
    sel = s["sel"]
    int4 = (sel["scale"].double() ** 2 * (sel["fmap"] >= 0)).sum() / 12 * T
    predicted = float((int4 + (0.02 * want_y.norm()) ** 2).sqrt() / want_y.norm())
    got = X.relative_error(y, want_y)
    say(f"  y {got:.4f} (predicted {predicted:.4f}), residual "
        f"{X.relative_error(residual, want_r):.4f}, z {X.relative_error(z, want_z):.4f}")
    assert got <= 1.5 * predicted
    # gate below 1 and unit-variance terms: the residual is no further off than
    # y's direction, and z not much further than the residual
    assert X.relative_error(residual, want_r) <= 2 * got
    assert X.relative_error(z, want_z) <= 2 * got + 0.04
    # the same calls again, and on another stream, give the same bits
    for a, b in zip((y, residual, z), X.step(s)):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = X.step(s)
    side.synchronize()
    for a, b in zip((y, residual, z), again):
        assert torch.equal(a, b)


def test_step_in_a_graph():
    say("case: tensor-parallel block captured in a graph, 3 replays")
    s = X.prepare(8, 16, 1024, 512, 256, 32)
    inputs = [(torch.randn_like(s["x"]), torch.randn_like(s["residual"])) for _ in range(3)]
    want = []
    for x, r in inputs:
        s["x"].copy_(x)
        s["residual"].copy_(r)
        want.append([t.clone() for t in X.step(s)])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = X.step(s)
    for (x, r), w in zip(inputs, want):
        s["x"].copy_(x)
        s["residual"].copy_(r)
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, w):
            assert torch.equal(a, b)
