"""btq_block_norm against plain numpy in 64 bits.

Tolerances are first-order bounds on the fp32 arithmetic, carried through the
formula (`bound_norm`): u = 2^-24 is one rounding, and a sum of H terms, added
in runs of at most H/64 and then pairwise, is off by at most
c = (H/64 + 16)*u of the sum of magnitudes. On top come the output's own
rounding (u for fp32, 2^-8 for bf16, half a step for 8-bit codes) and a
factor 1.05 for the terms of second order.
"""
import numpy as np
import pytest
import torch

import bit_tensor_activation_amd as B
from bit_tensor_activation_amd import _lib
from helpers import say

DEV = torch.device("cuda:0")
U = 2.0 ** -24
BF16, F32, I8 = torch.bfloat16, torch.float32, torch.int8


def host(t):
    if t is None:
        return None
    if t.dtype == torch.int16:
        t = t.view(BF16)
    return t.detach().double().cpu().numpy()


def bound_norm(v, ev, kind, weight, bias, eps):
    """(norm(v) in 64 bits, bound on the fp32 result's error) for inputs off by ev."""
    if kind == "none":
        return v, ev
    H = v.shape[-1]
    c = (H / 64 + 16) * U
    w = 1.0 if weight is None else weight
    if kind == "layer":
        mean = v.mean(-1, keepdims=True)
        em = ev.mean(-1, keepdims=True) + c * np.abs(v).mean(-1, keepdims=True) + U * np.abs(mean)
        d = v - mean
        ed = ev + em + U * np.abs(d)
    else:
        d, ed = v, ev
    ms = (d * d).mean(-1, keepdims=True) + eps
    rel = 0.5 * (c + 3 * U) + (np.abs(d) * ed + ed * ed).mean(-1, keepdims=True) / ms + 2 * U
    out = d / np.sqrt(ms) * w
    err = np.abs(w) / np.sqrt(ms) * ed + np.abs(out) * (rel + 2 * U)
    if bias is not None:
        out = out + bias
        err = err + U * np.abs(out)
    return out, err


def plain(y, residual, post, pw, pb, gate, alpha, pre, nw, nb, eps, post_eps):
    """(r', its bound, n, its bound)."""
    r, er = residual, np.zeros_like(residual)
    if y is not None:
        u, eu = bound_norm(y, np.zeros_like(y), post, pw, pb, post_eps)
        if gate is not None:
            g = np.repeat(gate, u.shape[0] // gate.shape[0], 0)
            u, eu = u * g, eu * np.abs(g) + U * np.abs(u * g)
        a = float(np.float32(alpha))
        r = residual + a * u
        er = np.abs(a) * eu + U * np.abs(a * u) + U * np.abs(r)
    n, en = bound_norm(r, er, pre, nw, nb, eps)
    return r, er, n, en


ROUND = {F32: U, BF16: 2.0 ** -8, torch.int16: 2.0 ** -8}


def within(got, want, err, dtype, what):
    tol = 1.05 * err + ROUND[dtype] * np.abs(want) + 2.0 ** -133
    off = np.abs(host(got) - want)
    assert (off <= tol).all(), (f"{what}: {(off > tol).sum()} of {off.size} off, worst "
                                f"{np.max(off - tol)} at {np.argwhere(off > tol)[0]}")


def check(T, H, y_dt=F32, r_dt=BF16, n_dt=BF16, post="rms", pre="rms", gate=None, G=1, alpha=1.0,
          weights=True, eps=1e-6, post_eps=None, seed=0, make=None, inplace=False):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + T * 1009 + H)

    def rnd(*shape):
        return torch.randn(shape, generator=g, device=DEV)
    y = None if y_dt is None else (rnd(T, H) * 3 + 0.5).to(y_dt)
    residual = (rnd(T, H) * 2 - 0.25).to(r_dt)
    if make is not None:
        make(y, residual)
    kw = dict(post=post if y is not None else "none", pre=pre, alpha=alpha, eps=eps,
              post_eps=post_eps)
    if weights and kw["post"] != "none":
        kw["post_weight"] = 1 + 0.3 * rnd(H)
    if weights and pre != "none":
        kw["pre_weight"] = 1 + 0.3 * rnd(H)
    if weights and kw["post"] == "layer":
        kw["post_bias"] = rnd(H)
    if weights and pre == "layer":
        kw["pre_bias"] = rnd(H)
    if gate is not None and y is not None:
        kw["gate"] = rnd(G, H).to(gate)
    r64, er, n64, en = plain(
        host(y), host(residual), kw["post"], host(kw.get("post_weight")), host(kw.get("post_bias")),
        host(kw.get("gate")), alpha, pre, host(kw.get("pre_weight")), host(kw.get("pre_bias")),
        float(np.float32(eps)), float(np.float32(eps if post_eps is None else post_eps)))
    if inplace:
        residual = residual.clone()
    out = B.btq_block_norm(y, residual, n_dtype=n_dt, residual_out=residual if inplace else None,
                           **kw)
    within(out[0], r64, er, r_dt, "residual")
    if n_dt != I8:
        within(out[1], n64, en, n_dt, "n")
        return out
    codes, scale = out[1].cpu().numpy().astype(np.float64), host(out[2])
    m = np.abs(n64).max(-1)
    dm = 1.05 * en.max(-1) + 2 * U * m
    assert (np.abs(scale * 127 - m) <= dm)[m > 1e-30].all(), "n_scale"
    step = scale[:, None]
    off = np.abs(codes * step - n64)
    tol = step * (0.5 + 127 * 2.0 ** -20) + 1.05 * en
    assert (off <= tol).all(), f"codes: worst {np.max(off - tol)}"
    assert np.abs(codes).max(-1).min() == 127
    return out


SIZES = [(1, 1), (1, 2), (2, 7), (3, 8), (5, 63), (4, 64), (1, 65), (7, 100), (3, 256), (2, 504),
         (9, 512), (3, 520), (1, 1000), (3, 1001), (6, 1024), (2, 1032), (33, 2048), (2, 2056),
         (1, 4096), (65, 4096), (300, 4096), (2, 5000), (1, 8192), (64, 8192), (2, 8200), (2, 9001),
         (1, 16384), (2, 16400), (1, 20000), (2, 32768), (1, 33000), (1, 65536), (1, 70001)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", SIZES)
def test_sizes(T, H):
    say(f"case: block norm T={T} H={H}")
    check(T, H)
    check(T, H, BF16, F32, F32, gate=F32, alpha=0.5)
    check(T, H, F32, F32, F32, post="layer", pre="layer", gate=BF16, G=T, alpha=-0.75)
    check(T, H, BF16, BF16, I8, post="layer", pre="rms")
    check(T, H, F32, BF16, I8, post="none", pre="layer", gate=F32, G=T)


@pytest.mark.gpu
@pytest.mark.parametrize("n_dt", [F32, BF16, I8])
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("T,H", [(6, 72), (6, 333), (4, 2048)])
def test_kinds_and_types(T, H, post, pre, n_dt):
    say(f"case: block norm {post}/{pre} n={n_dt} T={T} H={H}")
    for y_dt in (F32, BF16, None):
        for r_dt in (F32, BF16):
            check(T, H, y_dt, r_dt, n_dt, post, pre)
            check(T, H, y_dt, r_dt, n_dt, post, pre, weights=False, gate=BF16, G=2, alpha=2.0,
                  eps=1e-3, post_eps=1e-2, inplace=True)


@pytest.mark.gpu
@pytest.mark.parametrize("G", [1, 2, 3, 4, 6, 12])
@pytest.mark.parametrize("H", [256, 129])
def test_gate_rows(G, H):
    say(f"case: block norm gate rows G={G} H={H}")
    check(12, H, gate=F32, G=G, n_dt=F32, r_dt=F32)
    check(12, H, gate=BF16, G=G)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [64, 777, 8192, 40000])
def test_offset_rows_keep_their_variance(H):
    # a mean a thousand times the deviation: a one-pass sum of squares in fp32
    # would lose the variance; the deviations from the mean do not
    say(f"case: block norm rows with a large mean H={H}")

    def make(y, residual):
        y.add_(3000.0)
        residual.mul_(0.5).add_(1000.0)
    check(3, H, F32, F32, F32, "layer", "layer", make=make)


@pytest.mark.gpu
@pytest.mark.parametrize("H", [64, 1001, 4096])
def test_zero_and_constant_rows(H):
    say(f"case: block norm zero and constant rows H={H}")
    for post, pre in (("rms", "rms"), ("layer", "layer")):
        y = torch.zeros((3, H), device=DEV)
        r = torch.zeros((3, H), device=DEV)
        y[1], r[1] = 2.0, 0.0
        y[2], r[2] = 0.0, -4.0
        ro, n = B.btq_block_norm(y, r, post=post, pre=pre, n_dtype=F32)
        r64, er, n64, en = plain(host(y), host(r), post, None, None, None, 1.0, pre, None, None,
                                 float(np.float32(1e-6)), float(np.float32(1e-6)))
        within(ro, r64, er, F32, "residual")
        within(n, n64, en, F32, "n")
        _, q, s = B.btq_block_norm(y * 0, r * 0, post=post, pre=pre, n_dtype=I8)
        assert (q == 0).all() and (s == 1).all()
    # eps 0 on a row of zeros: 0 * (1/0) is NaN by the formula
    _, n = B.btq_block_norm(None, torch.zeros((1, H), device=DEV), eps=0.0, n_dtype=F32)
    assert torch.isnan(n).all()


@pytest.mark.gpu
@pytest.mark.parametrize("H", [64, 1001, 4096, 40000])
@pytest.mark.parametrize("n_dt", [F32, BF16, I8])
def test_nan_and_inf_stay_in_their_rows(H, n_dt):
    say(f"case: block norm NaN and Inf H={H} {n_dt}")
    y = torch.randn((5, H), device=DEV)
    r = torch.randn((5, H), device=DEV)
    y[1, H // 2] = float("nan")
    r[3, H - 1] = float("inf")
    for post, pre in (("rms", "rms"), ("layer", "layer"), ("none", "rms")):
        out = B.btq_block_norm(y, r, post=post, pre=pre, n_dtype=n_dt)
        ref = B.btq_block_norm(y[::2].contiguous(), r[::2].contiguous(), post=post, pre=pre,
                               n_dtype=n_dt)
        for a, b in zip(out, ref):
            assert torch.equal(a[::2], b), (post, pre)      # the clean rows
        if n_dt == I8:
            assert torch.isnan(out[2][[1, 3]]).all() and (out[1][[1, 3]] == 0).all()
        else:
            assert torch.isnan(out[1][1]).all()
            assert torch.isnan(out[1][3, H - 1])            # Inf * (1/Inf)
        assert torch.isinf(out[0][3, H - 1])


@pytest.mark.gpu
@pytest.mark.parametrize("H", [64, 200, 1001, 4096])
def test_alignment_and_guards(H):
    # every tensor off the vector boundary in turn; nothing around the outputs
    # is written
    say(f"case: block norm alignment H={H}")
    T = 3

    def at(t, off):
        buf = torch.full((t.numel() + 32,), 9, dtype=t.dtype, device=DEV)
        v = buf[off:off + t.numel()].view(t.shape)
        v.copy_(t)
        return v, buf
    for n_dt in (BF16, F32, I8):
        y = torch.randn((T, H), device=DEV)
        r = torch.randn((T, H), device=DEV).to(BF16)
        w, b = torch.randn(H, device=DEV), torch.randn(H, device=DEV)
        gate = torch.randn((T, H), device=DEV).to(BF16)
        kw = dict(post="layer", pre="layer")
        ref = B.btq_block_norm(y, r, post_weight=w, post_bias=b, pre_weight=b, pre_bias=w,
                               gate=gate, n_dtype=n_dt, **kw)
        for which in range(8):
            off = [1 if i == which else 0 for i in range(8)]
            ro, ro_buf = at(torch.zeros_like(r), off[4])
            n, n_buf = at(torch.zeros((T, H), dtype=n_dt, device=DEV), off[5])
            out = B.btq_block_norm(at(y, off[0])[0], at(r, off[1])[0],
                                   post_weight=at(w, off[2])[0], post_bias=at(b, off[6])[0],
                                   pre_weight=at(b, off[3])[0], pre_bias=w,
                                   gate=at(gate, off[7])[0], residual_out=ro, n=n, **kw)
            for a, c in zip(out, ref):
                d = (a.float() - c.float()).abs().max()
                assert d <= (1 if n_dt == I8 else 0.05), (which, d)   # another order of sums
            for buf, o in ((ro_buf, off[4]), (n_buf, off[5])):
                assert (buf[:o] == 9).all() and (buf[o + T * H:] == 9).all()


@pytest.mark.gpu
def test_same_bits_every_time_and_for_every_batch_size():
    # a row's result does not depend on the rows around it within one kernel
    # variant, and never on the run
    say("case: block norm repeatable")
    y = torch.randn((300, 4096), device=DEV)
    r = torch.randn((300, 4096), device=DEV).to(BF16)
    a = B.btq_block_norm(y, r, post="rms")
    for _ in range(3):
        b = B.btq_block_norm(y, r, post="rms")
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.gpu
def test_int8_output_feeds_the_product():
    say("case: block norm to 8 bits, then the product")
    T, H, P, N = 40, 512, 4, 96
    y, r = torch.randn((T, H), device=DEV), torch.randn((T, H), device=DEV).to(BF16)
    w, sw = B.btq_quantize_rows(torch.randn((P, N, H), device=DEV))
    _, n = B.btq_block_norm(y, r, post="rms", n_dtype=F32)
    _, q, s = B.btq_block_norm(y, r, post="rms", n_dtype=I8)
    q2, s2 = B.btq_quantize_rows(n)
    assert torch.equal(q, q2) and torch.equal(s, s2)       # the codes of the fp32 norm
    z = B.btq_int8_matmul(q, s, w, sw, bf16=False)
    assert torch.equal(z, B.btq_int8_linear(n, w, sw, bf16=False))


@pytest.mark.gpu
def test_large_rows_past_32_bit_offsets():
    say("case: block norm, more than 2^31 elements")
    T, H = (1 << 31) // 8192 + 5, 8192
    y = torch.empty((T, H), dtype=BF16, device=DEV)
    y.normal_()
    r = torch.zeros((T, H), dtype=BF16, device=DEV)
    r[T - 3:] = 1.0
    out = B.btq_block_norm(y, r, post="rms")
    for sl in (slice(0, 2), slice(T - 4, T)):
        r64, er, n64, en = plain(host(y[sl]), host(r[sl]), "rms", None, None, None, 1.0, "rms",
                                 None, None, float(np.float32(1e-6)), float(np.float32(1e-6)))
        within(out[0][sl], r64, er, BF16, "residual")
        within(out[1][sl], n64, en, BF16, "n")


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(1, 4096), (50, 1001)])
def test_side_stream_and_graph(T, H):
    say(f"case: block norm on a side stream and in a graph T={T} H={H}")
    ys = [torch.randn((T, H), device=DEV) for _ in range(4)]
    r = torch.randn((T, H), device=DEV).to(BF16)
    ref = [B.btq_block_norm(y, r, post="rms", n_dtype=I8) for y in ys]
    torch.cuda.synchronize()
    side = torch.cuda.Stream(device=DEV)   # default priority
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = [B.btq_block_norm(y, r, post="rms", n_dtype=I8, stream=side) for y in ys]
    junk = [torch.full((1 << 18,), -7, dtype=torch.int32, device=DEV) for _ in range(16)]
    side.synchronize()
    torch.cuda.synchronize()
    del junk
    for a, b in zip(ref, got):
        assert all(torch.equal(i, j) for i, j in zip(a, b))
    y, out = ys[0].clone(), [torch.empty_like(t) for t in ref[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.btq_block_norm(y, r, post="rms", residual_out=out[0], n=out[1], n_scale=out[2])
    for yi, want in zip(ys, ref):
        y.copy_(yi)
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(i, j) for i, j in zip(out, want))


@pytest.mark.gpu
def test_empty_batch_and_binding_refusals():
    say("case: block norm, empty batch and argument checks")
    e = torch.empty((0, 16), device=DEV)
    assert B.btq_block_norm(e, e, post="rms")[1].shape == (0, 16)
    y, r, w = torch.zeros((4, 16), device=DEV), torch.zeros((4, 16), device=DEV), torch.ones(
        16, device=DEV)
    for exc, call in (
            (ValueError, lambda: B.btq_block_norm(y, r, post="batch")),
            (ValueError, lambda: B.btq_block_norm(y[:2], r)),
            (ValueError, lambda: B.btq_block_norm(y, r.t())),
            (ValueError, lambda: B.btq_block_norm(y, r[0])),
            (TypeError, lambda: B.btq_block_norm(y.double(), r)),
            (TypeError, lambda: B.btq_block_norm(y, r, pre_weight=w.to(BF16))),
            (ValueError, lambda: B.btq_block_norm(y, r, pre_weight=w[:8])),
            (RuntimeError, lambda: B.btq_block_norm(y, r, pre_bias=w)),
            (RuntimeError, lambda: B.btq_block_norm(y, r, post_weight=w)),
            (RuntimeError, lambda: B.btq_block_norm(y, r, gate=torch.ones((3, 16), device=DEV))),
            (ValueError, lambda: B.btq_block_norm(y, r, gate=w)),
            (TypeError, lambda: B.btq_block_norm(y, r, residual_out=r.to(BF16))),
            (RuntimeError, lambda: B.btq_block_norm(None, r, post="rms")),
            (RuntimeError, lambda: B.btq_block_norm(y, r, eps=-1.0)),
            (RuntimeError, lambda: B.btq_block_norm(y, r, alpha=float("nan"))),
            (RuntimeError, lambda: B.btq_block_norm(y, r, n_scale=torch.ones(4, device=DEV))),
            (ValueError, lambda: B.btq_block_norm(y.cpu(), r))):
        with pytest.raises(exc):
            call()


A = 0x10000
OK, ARG, SHAPE, ALIGN = _lib.BTQ_OK, _lib.BTQ_ERR_ARG, _lib.BTQ_ERR_SHAPE, _lib.BTQ_ERR_ALIGN


def test_refusals():
    lib = _lib.load()
    nan, inf = float("nan"), float("inf")

    def call(y=A, yt=0, r=A, rt=1, T=4, H=16, post=1, pw=A, pb=None, pe=1e-6, gate=None, gt=0,
             gr=1, alpha=1.0, pre=1, nw=A, nb=None, ne=1e-6, ro=A, n=A, nt=1, ns=None):
        return lib.btq_block_norm(y, yt, r, rt, T, H, post, pw, pb, pe, gate, gt, gr, alpha, pre,
                                  nw, nb, ne, ro, n, nt, ns, None)
    for kw in (dict(H=0), dict(T=-1), dict(H=(1 << 30) + 1), dict(T=1 << 50, H=1 << 20),
               dict(gate=A, gr=3), dict(gate=A, gr=0), dict(gate=A, gr=8)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(post=3), dict(pre=-1), dict(yt=2), dict(rt=2), dict(gt=2), dict(nt=3),
               dict(pb=A), dict(nb=A), dict(post=0), dict(pre=0), dict(pe=-1.0), dict(ne=nan),
               dict(ne=inf), dict(alpha=inf), dict(alpha=nan), dict(r=None),
               dict(y=None), dict(y=None, post=0, pw=None, gate=A), dict(ro=None, n=None),
               dict(nt=2), dict(ns=A), dict(n=None, ns=A)):
        assert call(**kw) == ARG, kw
    for kw in (dict(y=A + 2), dict(y=A + 1, yt=1), dict(r=A + 1), dict(ro=A + 1), dict(n=A + 1),
               dict(n=A + 2, nt=0), dict(pw=A + 2), dict(nw=A + 1), dict(gate=A + 2),
               dict(nt=2, ns=A + 2), dict(post=2, pb=A + 1), dict(pre=2, nb=A + 2)):
        assert call(**kw) == ALIGN, kw
    assert call(T=0, y=None, r=None, ro=None, n=None, post=0, pw=None) == OK
