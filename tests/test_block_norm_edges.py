"""btq_block_norm where the last lanes of a row have nothing to hold, and where
a wide bound would hide it: norms with and without each of their weights,
constant rows with exact or tightly bounded results.

Bounds are those of test_block_norm (first-order, carried through the formula).
A bound near the size of what it checks would pass anything, so the tests also
assert how large it may be.
"""
import itertools

import numpy as np
import pytest
import torch

import bit_tensor_activation_amd as B
from helpers import say
from test_block_norm import BF16, DEV, F32, I8, ROUND, U, host, plain, within

pytestmark = pytest.mark.gpu


def rand(seed, *shape):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV)


def check_int8(q, s, n64, en, what):
    """Codes within half a step and n's own bound of the 64-bit n."""
    step = host(s)[:, None]
    m = np.abs(n64).max(-1)
    assert (np.abs(host(s) * 127 - m) <= 1.05 * en.max(-1) + 2 * U * m).all(), f"{what}: n_scale"
    off = np.abs(host(q) * step - n64)
    tol = step * (0.5 + 127 * 2.0 ** -20) + 1.05 * en
    assert (off <= tol).all(), f"{what}: codes off by {np.max(off - tol)}"


@pytest.mark.parametrize("post", ["rms", "layer"])
@pytest.mark.parametrize("H", [72, 333, 512, 1001, 2560, 5000, 5120, 9001, 17000])
def test_each_weight_present_or_absent(H, post):
    # y's mean is twice its deviation: lanes past H that held anything but 0
    # after the first norm would show in the second one's sums
    T = 3
    y32, r32 = rand(H, T, H) + 2.0, rand(H + 1, T, H) * 0.5
    w, b, gate = 1 + 0.3 * rand(H + 2, H), rand(H + 3, H), rand(H + 4, 1, H)
    for dt in (F32, BF16):
        y, r = y32.to(dt), r32.to(dt)
        for pw, pb, gt, pre, nw in itertools.product(
                (None, w), (None, b) if post == "layer" else (None,), (None, gate),
                ("rms", "layer", "none"), (None, w)):
            if pre == "none" and nw is not None:
                continue
            nb = b if pre == "layer" and nw is not None else None
            what = (f"block norm {post}/{pre} H={H} {dt} weight={pw is not None} "
                    f"bias={pb is not None} gate={gt is not None} pre weight={nw is not None}")
            say(f"case: {what}")
            r64, er, n64, en = plain(host(y), host(r), post, host(pw), host(pb), host(gt), -0.5,
                                     pre, host(nw), host(nb), float(np.float32(1e-6)),
                                     float(np.float32(1e-6)))
            # tight enough to see one foreign term in a hundred
            assert np.max(en) < 5e-3
            kw = dict(post=post, post_weight=pw, post_bias=pb, gate=gt, alpha=-0.5, pre=pre,
                      pre_weight=nw, pre_bias=nb)
            for n_dt in (F32, BF16, I8):
                out = B.btq_block_norm(y, r, n_dtype=n_dt, **kw)
                within(out[0], r64, er, dt, f"{what}: residual")
                if n_dt == I8:
                    check_int8(out[1], out[2], n64, en, what)
                else:
                    within(out[1], n64, en, n_dt, f"{what}: n")


@pytest.mark.parametrize("H", [64, 128, 256, 512, 1024, 4096, 65536])
@pytest.mark.parametrize("weights", [False, True])
def test_constant_rows_are_exact(H, weights):
    # sums of twos and a division by a power of two are exact, so a layer
    # norm's deviations are 0 and its result is 0, or its bias
    say(f"case: block norm, layer norm of constant rows H={H} weights={weights}")
    y = torch.full((3, H), 2.0, device=DEV)
    r = torch.zeros((3, H), device=DEV)
    kw = dict(post_weight=1 + rand(H, H), pre_weight=1 + rand(H + 1, H)) if weights else {}
    for pre in ("rms", "layer", "none"):
        if pre == "none":
            kw.pop("pre_weight", None)
        ro, n = B.btq_block_norm(y, r, post="layer", pre=pre, n_dtype=F32, **kw)
        assert (ro == 0).all() and (n == 0).all(), pre
        _, q, s = B.btq_block_norm(y, r, post="layer", pre=pre, n_dtype=I8, **kw)
        assert (q == 0).all() and (s == 1).all(), pre


@pytest.mark.parametrize("H", [72, 1001, 5000, 33001])
def test_constant_rows_of_any_length(H):
    # eps of 1e-2 keeps what the first norm's rounding becomes in the second
    # far below 1
    say(f"case: block norm, layer norm of constant rows H={H}")
    y = torch.full((3, H), 2.0, device=DEV)
    r = torch.zeros((3, H), device=DEV)
    eps = float(np.float32(1e-2))
    for pre in ("rms", "layer"):
        r64, er, n64, en = plain(host(y), host(r), "layer", None, None, None, 1.0, pre, None, None,
                                 eps, eps)
        assert np.max(er) < 1e-2 and np.max(en) < 0.1
        ro, n = B.btq_block_norm(y, r, post="layer", pre=pre, eps=1e-2, n_dtype=F32)
        within(ro, r64, er, F32, "residual")
        within(n, n64, en, F32, "n")


@pytest.mark.parametrize("dt", [F32, BF16])
def test_large_constant_rows(dt):
    # mean * 1/sqrt(eps) passes the largest fp32, the deviations are 0: the row
    # is its bias, and no Inf of an empty lane may meet its zero weight
    say(f"case: block norm, layer norm of rows of 2^120 {dt}")
    H = 64
    y = torch.full((2, H), 2.0 ** 120, device=DEV).to(dt)
    r = rand(1, 2, H).to(dt)
    w, b = 1 + 0.3 * rand(2, H), rand(3, H)
    for pre in ("rms", "layer"):
        kw = dict(pre=pre, pre_weight=w, n_dtype=F32)
        ro, n = B.btq_block_norm(y, r, post="layer", post_weight=w, post_bias=b, **kw)
        r64 = host(r) + host(b)
        within(ro, r64, U * np.abs(r64), dt, "residual")
        r64, er, n64, en = plain(None, r64, "none", None, None, None, 1.0, pre, host(w), None,
                                 float(np.float32(1e-6)), float(np.float32(1e-6)))
        # r' carries one rounding into n: of the row's norm, sqrt(H) at most
        within(n, n64, en + 4 * U * np.sqrt(H) * np.abs(host(w)), F32, "n")


@pytest.mark.parametrize("H", [40000, (1 << 22) + 3])
def test_long_rows_keep_their_sums(H):
    # Rows past the register kernels. Near-constant values make every rounding
    # of a running fp32 sum fall the same way: H/256 of them one after another
    # would be off by far more than the bound, which allows the sums only the
    # rounding of their result. n = v * rstd: var + eps, its root, the
    # quotient and the product round once each, and so does var (half of that in
    # rstd): 4.5 roundings, and the first order of it. A layer norm's mean
    # rounds too: the deviations move by U*|mean|, their own rounding by U*|d|.
    say(f"case: block norm, long rows H={H}")
    v = (0.7 + 0.01 * rand(H, 2, H)).to(F32)
    x = host(v)
    _, n = B.btq_block_norm(None, v, pre="rms", n_dtype=F32)
    want = x / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(1e-6)))
    off = np.abs(host(n) - want)
    assert (off <= 6 * U * np.abs(want)).all(), f"rms: off by {np.max(off / np.abs(want)) / U} u"
    _, n = B.btq_block_norm(None, v, pre="layer", n_dtype=F32)
    mean = x.mean(-1, keepdims=True)
    d = x - mean
    rstd = 1 / np.sqrt((d * d).mean(-1, keepdims=True) + float(np.float32(1e-6)))
    off = np.abs(host(n) - d * rstd)
    tol = (2 * U * np.abs(mean) + 8 * U * np.abs(d)) * rstd
    assert (off <= tol).all(), f"layer: off by {np.max(off)}, at most {np.max(tol)} allowed"
    # the same through the first norm, whose weights are absent
    _, n2 = B.btq_block_norm(v, torch.zeros_like(v), post="layer", pre="none", n_dtype=F32)
    assert torch.equal(n2, n)


@pytest.mark.parametrize("H", [72, 1001, 5000, 8192, 33000])
def test_second_norm_weight_or_bias_alone(H):
    T = 3
    y, r = rand(H, T, H) + 2.0, rand(H + 1, T, H) * 0.5
    w, b = 1 + 0.3 * rand(H + 2, H), rand(H + 3, H)
    eps = float(np.float32(1e-6))
    for nw, nb in ((None, None), (w, None), (None, b), (w, b)):
        say(f"case: block norm layer/layer H={H} pre weight={nw is not None} "
            f"bias={nb is not None}")
        r64, er, n64, en = plain(host(y), host(r), "layer", None, None, None, 1.0, "layer",
                                 host(nw), host(nb), eps, eps)
        assert np.max(en) < 1e-2
        for n_dt in (F32, I8):
            out = B.btq_block_norm(y, r, post="layer", pre="layer", pre_weight=nw, pre_bias=nb,
                                   n_dtype=n_dt)
            within(out[0], r64, er, F32, "residual")
            if n_dt == I8:
                check_int8(out[1], out[2], n64, en, "pre weight or bias alone")
            else:
                within(out[1], n64, en, F32, "n")


@pytest.mark.parametrize("r_dt", [F32, BF16])
@pytest.mark.parametrize("H", [200, 1000, 1001, 1024, 2047, 4096, 5000, 5001, 8192, 20000, 33000])
def test_rows_do_not_depend_on_the_batch(H, r_dt):
    # a row alone, in a few, in many: bit for bit, within a kernel variant
    # (4096 < H <= 8192 changes its lanes at T = 256)
    T = 300
    y, r = rand(H, T, H) + 1.0, rand(H + 1, T, H).to(r_dt)
    w = 1 + 0.3 * rand(H + 2, H)

    def run(rows, n_dt):
        return B.btq_block_norm(y[rows].contiguous(), r[rows].contiguous(), post="layer",
                                post_weight=w, pre="rms", n_dtype=n_dt)
    for n_dt in (F32, BF16, I8):
        say(f"case: block norm rows in other batches H={H} {r_dt} {n_dt}")
        if 4096 < H <= 8192:
            few, many = (slice(0, 256), (slice(0, 1), slice(0, 7), slice(100, 137))), (
                slice(0, 300), (slice(0, 257), slice(20, 290)))
            groups = (few, many)
        else:
            groups = ((slice(0, 300), (slice(0, 1), slice(0, 7), slice(100, 137), slice(1, 300))),)
        for whole, parts in groups:
            ref = run(whole, n_dt)
            for p in parts:
                at = slice(p.start - whole.start, p.stop - whole.start)
                for a, c in zip(run(p, n_dt), ref):
                    assert torch.equal(a, c[at]), (p, n_dt)


@pytest.mark.parametrize("T,H", [((1 << 22) + 5, 8), ((1 << 20) + 7, 1032)])
def test_more_rows_than_blocks(T, H):
    # a block then takes several rows, one after another, and the sums of one
    # must not meet the next one's
    say(f"case: block norm and codes of T={T} H={H}")
    y = torch.empty((T, H), dtype=BF16, device=DEV).normal_(1.0, 1.0)
    r = torch.empty((T, H), dtype=BF16, device=DEV).normal_()
    kw = dict(post="layer", pre="layer", n_dtype=I8)
    whole = B.btq_block_norm(y, r, **kw)
    codes = B.btq_quantize_rows(y)
    for sl in (slice(0, 9), slice((1 << 20) - 3, (1 << 20) + 7), slice(T - 1040, T)):
        for a, b in zip(B.btq_block_norm(y[sl].contiguous(), r[sl].contiguous(), **kw), whole):
            assert torch.equal(a, b[sl])
        for a, b in zip(B.btq_quantize_rows(y[sl]), codes):
            assert torch.equal(a, b[sl])
    # every row, by its codes' scale: the largest |code| of a row is 127
    assert (whole[1].abs().amax(-1) == 127).all() and torch.isfinite(whole[2]).all()
