"""btq_head_norm_rope against plain numpy in 64 bits.

Tolerance: a sum of D terms in fp32 is off by at most c = (D/64 + 16)*U of the sum
of magnitudes (U = 2^-24; runs of at most D/64 and then pairs, 16 to a lane and
pairs in the vector kernel), so the norm is off by rel = (c + 8)*U-sized steps as
carried below; a rotation adds two products and a sum. The output's own rounding
is U (fp32) or 2^-8 (bf16). A factor 1.05 covers terms of second order.
"""
import numpy as np
import pytest
import torch

import bit_tensor_activation_amd as B
from bit_tensor_activation_amd import _lib
from helpers import say
from kv_helpers import BF16, DEV, F32, U, host, table, turn

EPS = 1e-6
ROUND = {F32: U, BF16: 2.0 ** -8, torch.int16: 2.0 ** -8}


def plain(x, qh, norm, qw, kw, pos, cos, sin, style):
    """(y, bound) [P,T,H,D]."""
    D = x.shape[-1]
    c = (D / 64 + 16 + min(D, 16)) * U
    err = np.zeros_like(x)
    if norm == "layer":
        em = c * np.abs(x).mean(-1, keepdims=True) + U * np.abs(x.mean(-1, keepdims=True))
        x = x - x.mean(-1, keepdims=True)
        err = em + U * np.abs(x)
    if norm != "none":
        ms = (x * x).mean(-1, keepdims=True) + float(np.float32(EPS))
        rel = 0.5 * (c + 3 * U) + (np.abs(x) * err + err * err).mean(-1, keepdims=True) / ms + 4 * U
        err = err / np.sqrt(ms) + np.abs(x) / np.sqrt(ms) * rel
        x = x / np.sqrt(ms)
    w = np.ones(x.shape[-2:])[None, None].repeat(x.shape[0], 0)
    for part, v in ((slice(0, qh), qw), (slice(qh, None), kw)):
        if v is not None:
            v = host(v)
            w[:, 0, part] = v if v.ndim < 3 else v
    err = err * np.abs(w) + U * np.abs(x * w) * (qw is not None or kw is not None)
    x = x * w
    if cos is not None:
        cs, sn = host(cos)[pos][:, None], host(sin)[pos][:, None]
        turned = turn(err, np.abs(cs), np.abs(sn), style)     # second feature: sums
        other = turn(err, np.abs(cs), -np.abs(sn), style)     # first feature: sums
        big = np.maximum(turn(np.abs(x), np.abs(cs), np.abs(sn), style),
                         turn(np.abs(x), np.abs(cs), -np.abs(sn), style))
        err = np.maximum(turned, other)
        n = 2 * cos.shape[-1]
        err[..., :n] += 2 * U * big[..., :n]
        x = turn(x, cs, sn, style)
    return x, err


def within(got, want, err, dtype):
    tol = 1.05 * err + ROUND[dtype] * np.abs(want) + 2.0 ** -133
    off = np.abs(host(got) - want)
    assert (off <= tol).all(), (f"{(off > tol).sum()} of {off.size} off, worst {np.max(off - tol)} "
                                f"at {np.argwhere(off > tol)[0]}")


def check(P, T, Hq, Hk, D, dim=0, style="half", norm="rms", x_dt=BF16, y_dt=BF16, weights="one",
          inplace=False, shift=0, gap=0, rows=97):
    g = torch.Generator(device=DEV)
    g.manual_seed(P * 7919 + T * 131 + Hq * 17 + Hk * 5 + D)

    def rnd(*shape):
        return torch.randn(shape, generator=g, device=DEV)
    H = Hq + Hk
    size = P * T * (H * D + gap) + shift
    flat = (rnd(size) * 2 + 0.25).to(x_dt)
    x = flat[shift:].view(P, T, H * D + gap)[..., :H * D].unflatten(-1, (H, D))
    qw = kw = None
    if weights == "one":
        qw, kw = 1 + 0.3 * rnd(D), 1 + 0.3 * rnd(D)
    elif weights == "heads":
        qw, kw = 1 + 0.3 * rnd(P, Hq, D), 1 + 0.3 * rnd(P, Hk, D)
    cos = sin = pos = None
    if dim:
        cos, sin = table(rows, dim)
        pos = torch.randint(0, rows, (T,), generator=g, device=DEV).int()
    want, err = plain(host(x), Hq, norm, qw, kw, None if pos is None else pos.cpu().numpy(), cos,
                      sin, style)
    guard = flat.clone()
    out = x if inplace else torch.empty((P, T, H, D), dtype=y_dt, device=DEV)
    got = B.btq_head_norm_rope(x, Hq, norm=norm, q_weight=qw, k_weight=kw, eps=EPS, positions=pos,
                               cos=cos, sin=sin, rope=style, out=out)
    assert got is out
    within(got, want, err, got.dtype)
    if inplace:                       # nothing between the heads has changed
        got = got.clone()
        x.copy_(guard[shift:].view(P, T, H * D + gap)[..., :H * D].unflatten(-1, (H, D)))
    assert torch.equal(flat.view(torch.int16), guard.view(torch.int16)), "input changed"
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("D", [1, 2, 3, 8, 16, 32, 48, 64, 80, 96, 100, 128, 192, 256, 257, 512,
                               1000, 1024, 1040, 4096])
def test_sizes(D):
    say(f"case: head norm D={D}")
    for norm in ("rms", "layer", "none"):
        check(2, 5, 3, 2, D, norm=norm)
        even = D // 2 * 2
        if even:
            check(1, 7, 2, 1, D, dim=even, norm=norm)
            check(1, 3, 4, 0, D, dim=even, style="pairs", norm=norm, x_dt=F32)
            check(2, 1, 0, 3, D, dim=max(2, even // 4 * 2), norm=norm, y_dt=F32)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 2, 31, 64, 300])
@pytest.mark.parametrize("x_dt,y_dt", [(BF16, BF16), (BF16, F32), (F32, BF16), (F32, F32)])
def test_rows_and_types(T, x_dt, y_dt):
    for style in ("half", "pairs"):
        check(8, T, 8, 1, 128, dim=128, style=style, x_dt=x_dt, y_dt=y_dt)
        check(3, T, 5, 2, 96, dim=64, style=style, norm="layer", x_dt=x_dt, y_dt=y_dt,
              weights="heads")


@pytest.mark.gpu
@pytest.mark.parametrize("shift,gap", [(0, 0), (0, 128), (0, 7), (1, 0), (3, 5), (8, 8)])
def test_strides_alignment_and_in_place(shift, gap):
    for x_dt in (BF16, F32):
        for D, dim in ((128, 128), (64, 32), (24, 6)):
            check(2, 9, 3, 2, D, dim=dim, x_dt=x_dt, shift=shift, gap=gap, y_dt=x_dt)
            check(2, 9, 3, 2, D, dim=dim, x_dt=x_dt, shift=shift, gap=gap, inplace=True,
                  style="pairs", weights=None)


@pytest.mark.gpu
def test_same_bits_in_other_batches_and_places():
    a = check(1, 300, 4, 2, 128, dim=128)
    again = check(1, 300, 4, 2, 128, dim=128)
    assert torch.equal(a, again)
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn((64, 6, 128), generator=g, device=DEV).to(BF16)
    cos, sin = table(64, 128)
    pos = torch.arange(64, dtype=torch.int32, device=DEV)
    whole = B.btq_head_norm_rope(x, 4, positions=pos, cos=cos, sin=sin)
    for t in (0, 31, 63):
        one = B.btq_head_norm_rope(x[t:t + 1], 4, positions=pos[t:t + 1], cos=cos, sin=sin)
        assert torch.equal(one[0], whole[t])


@pytest.mark.gpu
@pytest.mark.parametrize("D", [128, 100])
def test_positions_outside_the_table_turn_to_nan(D):
    x = torch.randn((6, 2, D), device=DEV)
    cos, sin = table(10, 32)
    pos = torch.tensor([0, 9, 10, -1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV)
    y = B.btq_head_norm_rope(x, 1, norm="none", positions=pos, cos=cos, sin=sin)
    assert torch.isfinite(y[:2]).all()
    assert torch.isnan(y[2:, :, :32]).all()
    assert torch.equal(y[2:, :, 32:], x[2:, :, 32:])


@pytest.mark.gpu
@pytest.mark.parametrize("D", [128, 100])
def test_nan_inf_zero_and_large_heads_stay_in_their_head(D):
    x = torch.randn((1, 8, D), device=DEV)
    ref = B.btq_head_norm_rope(x, 8)
    y = x.clone()
    y[0, 1, 3] = float("nan")
    y[0, 2, 0] = float("inf")
    y[0, 3] = 0
    y[0, 4] = 1e-30
    got = B.btq_head_norm_rope(y, 8)
    assert torch.isnan(got[0, 1]).all()
    assert torch.isnan(got[0, 2, 0]) and (got[0, 2, 1:] == 0).all()
    assert (got[0, 3] == 0).all()
    assert torch.allclose(got[0, 4], torch.full((D,), 1e-27, device=DEV), rtol=1e-5)
    assert torch.equal(got[0, 5:], ref[0, 5:]) and torch.equal(got[0, 0], ref[0, 0])


@pytest.mark.gpu
@pytest.mark.parametrize("T", [(1 << 20) + 1, (1 << 22) + 1])
def test_many_heads(T):
    # 2^25 heads of a shard and more go to the general kernel
    H, D = 8, 16
    x = torch.randn((T, H, D), device=DEV, dtype=F32).to(BF16)
    y = B.btq_head_norm_rope(x, H, norm="rms")
    assert torch.equal(y[-1:], B.btq_head_norm_rope(x[-1:].contiguous(), H))
    v = x.double()
    want = v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS)
    assert ((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-5).all()


@pytest.mark.gpu
def test_empty_batch():
    x = torch.empty((0, 3, 64), device=DEV, dtype=BF16)
    assert B.btq_head_norm_rope(x, 2).shape == (0, 3, 64)


@pytest.mark.gpu
def test_python_refusals():
    x = torch.zeros((4, 3, 64), device=DEV, dtype=BF16)
    cos, sin = table(8, 64)
    pos = torch.zeros(4, dtype=torch.int32, device=DEV)
    bad = [dict(norm="l2"), dict(rope="spiral"), dict(cos=cos, positions=pos),
           dict(cos=cos, sin=sin), dict(cos=cos, sin=sin[:4], positions=pos),
           dict(cos=cos, sin=sin, positions=pos[:3]),
           dict(q_weight=torch.ones(32, device=DEV)),
           dict(out=torch.zeros((4, 3, 32), device=DEV, dtype=BF16))]
    for kw in bad:
        with pytest.raises(ValueError):
            B.btq_head_norm_rope(x, 2, **kw)
    for kw in (dict(cos=cos, sin=sin, positions=pos.long()), dict(q_weight=torch.ones(64, device=DEV).double()),
               dict(out=torch.zeros((4, 3, 64), device=DEV, dtype=torch.float16))):
        with pytest.raises(TypeError):
            B.btq_head_norm_rope(x, 2, **kw)
    with pytest.raises(TypeError):
        B.btq_head_norm_rope(x.half(), 2)
    for q_heads in (-1, 4):
        with pytest.raises(ValueError):
            B.btq_head_norm_rope(x, q_heads)
    with pytest.raises(ValueError):
        B.btq_head_norm_rope(x[..., ::2], 2)
    with pytest.raises(RuntimeError):
        B.btq_head_norm_rope(x, 2, cos=table(8, 66)[0], sin=table(8, 66)[1], positions=pos)
    with pytest.raises(RuntimeError):
        B.btq_head_norm_rope(x, 2, eps=-1.0)


@pytest.mark.gpu
def test_outputs_whose_heads_overlap_are_refused():
    x = torch.zeros((2, 4, 3, 64), device=DEV, dtype=BF16)
    y = torch.zeros((2, 4, 3, 64), device=DEV, dtype=BF16)
    for out in (y[:, :, :1].expand(2, 4, 3, 64), y[:, :1].expand(2, 4, 3, 64), y[:1].expand(2, 4, 3, 64),
                y.as_strided((2, 4, 3, 64), (768, 192, 32, 1))):
        with pytest.raises(RuntimeError):
            B.btq_head_norm_rope(x, 2, out=out)
    # an input may be expanded, and an output may lie in any order
    turned = torch.zeros((3, 2, 4, 80), device=DEV, dtype=BF16).permute(1, 2, 0, 3)[..., :64]
    B.btq_head_norm_rope(x[:, :, :1].expand(2, 4, 3, 64), 2, out=turned)


# ---- CPU: all return before any HIP call ---------------------------------------

A = 0x10000


def call(x=A, xt=1, xs=0, xp=384, xh=128, P=1, T=4, qh=2, kh=1, D=128, norm=1, qw=A, qws=0, qwh=0,
         kw=A, kws=0, kwh=0, eps=1e-6, pos=A, cos=A, sin=A, rows=16, dim=128, rope=0, y=A, yt=1,
         ys=0, yp=384, yh=128):
    return _lib.load().btq_head_norm_rope(x, xt, xs, xp, xh, P, T, qh, kh, D, norm, qw, qws, qwh,
                                          kw, kws, kwh, eps, pos, cos, sin, rows, dim, rope, y, yt,
                                          ys, yp, yh, None)


def test_refusals():
    ARG, SHAPE, ALIGN = _lib.BTQ_ERR_ARG, _lib.BTQ_ERR_SHAPE, _lib.BTQ_ERR_ALIGN
    assert call(T=0) == _lib.BTQ_OK
    for kw in (dict(P=0), dict(P=65536), dict(T=-1), dict(D=0), dict(D=65537), dict(qh=0, kh=0),
               dict(qh=-1), dict(kh=-1), dict(qh=65536), dict(xs=-1), dict(xp=-1), dict(xh=-1),
               dict(yp=-1), dict(dim=0), dict(dim=3), dict(dim=130), dict(rows=0),
               dict(P=2, xs=1 << 61), dict(yp=1 << 61), dict(qws=-1), dict(kwh=-1),
               dict(P=2, qws=1 << 61), dict(T=1 << 60)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(x=None), dict(y=None), dict(xt=2), dict(yt=2), dict(xt=-1), dict(norm=3),
               dict(norm=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
               dict(cos=None), dict(sin=None), dict(pos=None), dict(rope=2)):
        assert call(**kw) == ARG, kw
    for kw in (dict(x=A + 1), dict(y=A + 1), dict(xt=0, x=A + 2), dict(pos=A + 2), dict(cos=A + 2),
               dict(sin=A + 1), dict(qw=A + 2), dict(kw=A + 1)):
        assert call(**kw) == ALIGN, kw


def test_overlapping_outputs():
    SHAPE = _lib.BTQ_ERR_SHAPE
    # (inputs of the same strides are taken: they get as far as the null pointer)
    for n in (dict(s=0, p=384, h=128), dict(s=1536, p=0, h=128), dict(s=1536, p=384, h=0),
              dict(s=1536, p=384, h=127), dict(s=1536, p=383, h=128), dict(s=1535, p=384, h=128),
              dict(s=128, p=256, h=1023), dict(s=0, p=0, h=0)):
        assert call(P=2, xs=1536, ys=n["s"], yp=n["p"], yh=n["h"]) == SHAPE, n
        assert call(P=2, xs=n["s"], xp=n["p"], xh=n["h"], ys=1536, x=None) == _lib.BTQ_ERR_ARG, n
    for n in (dict(s=1536, p=384, h=128), dict(s=128, p=256, h=1024), dict(s=512, p=128, h=1024),
              dict(s=1 << 40, p=1 << 30, h=1 << 20)):
        assert call(P=2, xs=1536, ys=n["s"], yp=n["p"], yh=n["h"], y=None) == _lib.BTQ_ERR_ARG, n
    # strides of an axis of one do not count
    assert call(T=1, yp=0, y=None) == _lib.BTQ_ERR_ARG
    assert call(qh=1, kh=0, yh=0, yp=128, y=None) == _lib.BTQ_ERR_ARG
