"""The 8-bit linear layer: btq_quantize_rows, btq_int8_matmul and
btq_int8_linear against plain numpy in 64 bits.

Tolerances. Integer sums are exact, and the three (four with bias) fp32 steps
after them are single IEEE operations, so y is compared bit for bit with those
steps on the int64 sum, and, against the 64-bit product, within 4 fp32
roundings (each 2^-24 of a value no larger than |sum*scales| + |bias|) plus the
output's own (2^-24 for fp32, 2^-8 for bf16). Codes of bf16 rows are exact:
127*x/m in float64 is either a tie or at least 1e-5 of itself away from one.
Codes of fp32 rows are within 1/2 + 127*2^-20 of it: the multiplier is off by
less than 2^-20 of itself.
"""
import numpy as np
import pytest
import torch

import bit_tensor_activation_amd as B
from bit_tensor_activation_amd import _lib
from helpers import say

DEV = torch.device("cuda:0")
U = 2.0 ** -24


# ---- plain forms -------------------------------------------------------------

def codes64(x):
    """(codes, scale fp32) of float64 rows; m/127 is one fp32 division."""
    m = np.abs(x).max(-1)
    bad = ~np.isfinite(x).all(-1)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        scale = m.astype(np.float32) / np.float32(127)
    tiny = ~bad & (scale < np.float32(2.0 ** -126))
    scale = np.where(bad, np.float32(np.nan), np.where(tiny, np.float32(1), scale))
    zero = bad | tiny
    v = np.where(zero[..., None], 0.0, x) * 127.0 / np.where(zero, 1.0, m)[..., None]
    return np.trunc(v + np.copysign(0.5, v)).astype(np.int64), scale.astype(np.float32), v


def bf16_round(f):
    """fp32 -> bf16 -> fp32, nearest even; NaN kept."""
    u = np.ascontiguousarray(f, np.float32).view(np.uint32)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16 << 16).astype(np.uint32)
    return np.where(np.isnan(f), np.float32(np.nan), r.view(np.float32))


def product(a, sa, w, sw, bias=None, bf16=True):
    """y by the documented fp32 steps from the int64 sum, and the 64-bit value."""
    acc = np.matmul(a.astype(np.float64), w.astype(np.float64).swapaxes(-1, -2))   # < 2^53: exact
    with np.errstate(invalid="ignore", over="ignore"):
        y = acc.astype(np.float32) * sa[..., None] * sw[:, None, :]
        ex = acc * sa.astype(np.float64)[..., None] * sw.astype(np.float64)[:, None, :]
        mag = np.abs(ex)
        if bias is not None:
            y = y + bias[:, None, :]
            ex = ex + bias.astype(np.float64)[:, None, :]
            mag = mag + np.abs(bias[:, None, :])
    return (bf16_round(y) if bf16 else y), ex, mag


def f32(t):
    if t.dtype == torch.int16:
        t = t.view(torch.bfloat16)
    return t.detach().float().cpu().numpy()


def assert_product(y, a, sa, w, sw, bias=None, what=""):
    bf16 = y.dtype != torch.float32
    want, ex, mag = product(a, sa, w, sw, bias, bf16)
    got = f32(y)
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    assert same.all(), f"{what}: {(~same).sum()} of {same.size} differ, first {np.argwhere(~same)[0]}"
    fin = np.isfinite(ex)
    off = np.abs(got.astype(np.float64) - ex)[fin]
    tol = (4 * U * mag + (2.0 ** -8 if bf16 else U) * np.abs(ex) + 2.0 ** -133)[fin]
    assert (off <= tol).all(), f"{what}: off the 64-bit product by {np.max(off - tol)}"


def gen(seed):
    return np.random.default_rng(seed)


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def rand_codes(rng, shape, full=False):
    if full:
        return rng.integers(-128, 128, shape).astype(np.int8)
    return np.clip(np.rint(rng.standard_normal(shape) * 32), -127, 127).astype(np.int8)


def case(rng, P, T, N, K, full=False, bias=False):
    a, w = rand_codes(rng, (P, T, K), full), rand_codes(rng, (P, N, K), full)
    sa = (0.5 + rng.random((P, T))).astype(np.float32) * np.float32(0.01)
    sw = (0.5 + rng.random((P, N))).astype(np.float32) * np.float32(0.001)
    b = rng.standard_normal((P, N)).astype(np.float32) if bias else None
    return a, sa, w, sw, b


# ---- quantize_rows -------------------------------------------------------------

ROWS = [(1, 1, 1), (1, 1, 2), (1, 3, 7), (2, 5, 8), (1, 4, 15), (1, 4, 16), (1, 4, 17), (3, 7, 64),
        (1, 2, 127), (1, 9, 512), (2, 3, 1000), (1, 5, 1001), (1, 3, 2048), (1, 2, 4104),
        (1, 300, 256), (1, 2, 8192), (1, 2, 16392), (1, 2, 32768), (1, 1, 40001), (1, 1, 100000)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("P,T,K", ROWS)
def test_quantize_rows(P, T, K, dtype):
    say(f"case: quantize_rows P={P} T={T} K={K} {dtype}")
    rng = gen(K * 7 + T)
    x = (rng.standard_normal((P, T, K)) * 10.0 ** rng.uniform(-6, 6, (P, T, 1))).astype(np.float32)
    xt = dev(x)
    if dtype == "bf16":
        xt = xt.to(torch.bfloat16)
    q, s = B.btq_quantize_rows(xt)
    codes, scale, v = codes64(f32(xt).astype(np.float64))
    assert np.array_equal(s.cpu().numpy().view(np.uint32), scale.view(np.uint32))
    got = q.cpu().numpy().astype(np.int64)
    if dtype == "bf16":
        assert np.array_equal(got, codes)
    else:
        assert (np.abs(got - v) <= 0.5 + 127 * 2.0 ** -20).all()
    assert np.abs(got).max(-1).min() == 127


@pytest.mark.gpu
def test_quantize_rows_every_bf16_pair():
    # every finite bf16 magnitude against every mantissa of the row's largest
    # value, so every tie that bf16 rows can hold; both signs
    say("case: quantize_rows, every bf16 magnitude below each of 128 largest values")
    bits = np.arange(0, 0x7F80, dtype=np.uint32)
    vals = (bits << 16).view(np.float32)
    for e in (0x3F80, 0x0800, 0x7F00):
        tops = ((np.arange(128, dtype=np.uint32) + e) << 16).view(np.float32)
        x = np.where(vals[None, :] <= tops[:, None], vals[None, :], 0).astype(np.float32)
        x[:, ::2] *= -1
        x = np.concatenate([x, tops[:, None]], 1)
        xt = dev(x).to(torch.bfloat16)
        q, s = B.btq_quantize_rows(xt)
        codes, scale, _ = codes64(x.astype(np.float64))
        assert np.array_equal(s.cpu().numpy(), scale)
        assert np.array_equal(q.cpu().numpy().astype(np.int64), codes)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [5, 64, 1000, 9000])
def test_quantize_rows_special_rows(K, dtype):
    say(f"case: quantize_rows special rows K={K} {dtype}")
    x = torch.randn((10, K), device=DEV)
    x[0] = 0
    x[1, K - 1] = float("inf")
    x[2, 0] = float("nan")
    x[3] = 1e-38                      # m/127 below the smallest normal number
    x[4] = -0.0
    x[5] = 3e38
    x[6, 1:] = 0
    x[7, K // 2] = -float("inf")
    x[8] = 1.5e-36
    x = x.to(dtype)
    q, s = B.btq_quantize_rows(x)
    codes, scale, v = codes64(f32(x).astype(np.float64))
    got = q.cpu().numpy().astype(np.int64)
    if dtype == torch.bfloat16:
        assert np.array_equal(got, codes)
    else:
        assert (np.abs(got - v) <= 0.5 + 127 * 2.0 ** -20).all()
    s = s.cpu().numpy()
    assert np.isnan(s[[1, 2, 7]]).all() and np.isfinite(np.delete(s, [1, 2, 7])).all()
    assert np.array_equal(np.nan_to_num(s, nan=-1), np.nan_to_num(scale, nan=-1))
    assert (got[[0, 1, 2, 3, 4, 7]] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("K", [24, 64, 1000, 4096])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_rows_strides_and_alignment(K, dtype):
    # shards as column slices of one matrix, rows cut out of a wider one, a
    # start off every vector boundary, one set of rows for all shards
    say(f"case: quantize_rows strides K={K} {dtype}")
    P, T = 3, 5
    whole = torch.randn((T, P * K), device=DEV).to(dtype)
    x = whole.view(T, P, K).transpose(0, 1)
    q, s = B.btq_quantize_rows(x)
    q2, s2 = B.btq_quantize_rows(x.contiguous())
    assert torch.equal(q, q2) and torch.equal(s, s2) and q.is_contiguous()
    for off in (1, 3, 4, 8):
        y = torch.randn((T, K + 13), device=DEV).to(dtype)[:, off:off + K]
        q, s = B.btq_quantize_rows(y)
        q2, s2 = B.btq_quantize_rows(y.contiguous())
        assert torch.equal(q, q2) and torch.equal(s, s2)
    buf = torch.randint(-9, 9, (T * K + 64,), dtype=torch.int8, device=DEV)
    for off in (1, 4, 8, 16):
        keep = buf.clone()
        out = buf[off:off + T * K].view(T, K)
        q, s = B.btq_quantize_rows(y, q=out)
        assert torch.equal(q, q2)
        assert torch.equal(buf[:off], keep[:off]) and torch.equal(buf[off + T * K:],
                                                                  keep[off + T * K:])
    same = whole[:, :K].unsqueeze(0).expand(P, T, K)
    q, s = B.btq_quantize_rows(same)
    q2, s2 = B.btq_quantize_rows(whole[:, :K])
    for p in range(P):
        assert torch.equal(q[p], q2) and torch.equal(s[p], s2)


# ---- int8_matmul -------------------------------------------------------------

SIZES = [  # P, T, N, K
    (1, 1, 1, 1), (1, 1, 5, 3), (2, 1, 16, 16), (1, 1, 64, 64), (1, 2, 33, 48), (3, 1, 100, 128),
    (1, 3, 17, 80), (8, 1, 256, 1024), (2, 4, 48, 2048), (1, 5, 96, 4096), (2, 8, 130, 256),
    (1, 9, 64, 1040), (1, 15, 31, 100), (1, 16, 128, 512), (2, 16, 272, 528), (3, 17, 65, 96),
    (1, 31, 200, 64), (2, 32, 64, 4112), (1, 33, 64, 64), (1, 48, 80, 208), (2, 63, 130, 272),
    (1, 64, 64, 2048), (1, 64, 1024, 4096), (3, 65, 129, 144), (3, 77, 999, 1000), (1, 100, 256, 63),
    (2, 127, 255, 129), (1, 128, 128, 128), (1, 129, 257, 256), (2, 200, 312, 176),
    (1, 256, 256, 64), (1, 256, 256, 128), (2, 256, 512, 384), (1, 257, 300, 400),
    (1, 300, 511, 4096), (2, 512, 256, 16), (1, 513, 1025, 160), (1, 1000, 1000, 1000),
    (1, 2048, 512, 1024), (2, 770, 520, 8192), (1, 4096, 24, 256), (1, 24, 4096, 256)]


@pytest.mark.gpu
@pytest.mark.parametrize("P,T,N,K", SIZES)
def test_int8_matmul(P, T, N, K):
    say(f"case: int8_matmul P={P} T={T} N={N} K={K}")
    rng = gen(T * 1000 + N + K)
    full = (T + N) % 2 == 0
    a, sa, w, sw, b = case(rng, P, T, N, K, full=full, bias=True)
    da, dsa, dw, dsw, db = dev(a), dev(sa), dev(w), dev(sw), dev(b)
    for bf16 in (True, False):
        assert_product(B.btq_int8_matmul(da, dsa, dw, dsw, bf16=bf16), a, sa, w, sw,
                       what=f"bf16={bf16}")
    assert_product(B.btq_int8_matmul(da, dsa, dw, dsw, bias=db), a, sa, w, sw, b, "bias")
    # one set of rows for every shard
    y = B.btq_int8_matmul(da[0].contiguous(), dsa[0].contiguous(), dw, dsw, bias=db, bf16=False)
    assert_product(y, np.repeat(a[:1], P, 0), np.repeat(sa[:1], P, 0), w, sw, b, "shared rows")


LARGE = [  # P, T, N, K: what takes each tile size, whole and ragged, aligned and not
    (8, 2048, 2048, 1040), (4, 2000, 4088, 2064), (3, 1500, 3001, 1168), (1, 4096, 4096, 1152),
    (2, 2048, 4096, 300), (8, 1024, 2048, 512), (1, 1000, 4104, 1296), (8, 250, 1016, 2048),
    (1, 512, 4096, 2048), (1, 300, 4100, 784), (8, 100, 1024, 1024), (1, 256, 4096, 4096),
    (1, 90, 4096, 1024), (8, 60, 8192, 528), (8, 33, 8190, 400), (8, 30, 8192, 2176),
    (8, 7, 8200, 656), (4, 50, 4096, 1024), (1, 1024, 4095, 2047), (3, 2047, 1023, 513),
    (8, 64, 2047, 1001), (2, 500, 900, 18), (2, 60, 8192, 1040), (8, 16, 8200, 4112),
    (8, 64, 8192, 4096), (9, 10, 16384, 2048), (8, 2048, 2048, 2043), (1, 1024, 4096, 1021),
    (8, 300, 999, 1001), (1, 256, 4096, 1030), (2, 100, 1000, 1029), (1, 2, 4095, 4095)]


@pytest.mark.gpu
@pytest.mark.parametrize("P,T,N,K", LARGE)
def test_int8_matmul_large(P, T, N, K):
    # the sums in float64 on the GPU: exact below 2^53, whatever their order
    say(f"case: int8_matmul P={P} T={T} N={N} K={K}")
    g = torch.Generator(device=DEV)
    g.manual_seed(K)
    a = torch.randint(-128, 128, (P, T, K), device=DEV, generator=g, dtype=torch.int8)
    w = torch.randint(-128, 128, (P, N, K), device=DEV, generator=g, dtype=torch.int8)
    sa, sw = torch.rand((P, T), device=DEV, generator=g), torch.rand((P, N), device=DEV,
                                                                     generator=g)
    bias = torch.randn((P, N), device=DEV, generator=g)
    for b in (None, bias):
        for bf16 in (True, False):
            y = B.btq_int8_matmul(a, sa, w, sw, bias=b, bf16=bf16)
            for p in range(P):
                acc = a[p].double() @ w[p].double().t().contiguous()
                want = acc.float() * sa[p][:, None] * sw[p][None, :]
                if b is not None:
                    want = want + b[p][None, :]
                got = y[p].view(torch.bfloat16) if bf16 else y[p]
                assert torch.equal(got, want.to(got.dtype)), (p, bf16, b is not None)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 16, 40, 300])
def test_int8_matmul_largest_sums(T):
    # every product 2^14 and K at its limit, and a K of full tiles: the sums
    # pass 2^24 (fp32 rounds them) and come near 2^31
    for K in (131071, 131056, 65536):
        say(f"case: int8_matmul largest sums T={T} K={K}")
        a = np.full((1, T, K), -128, np.int8)
        w = np.full((1, 3, K), -128, np.int8)
        w[0, 1] = 127
        sa, sw = np.full((1, T), 0.5, np.float32), np.full((1, 3), 0.25, np.float32)
        y = B.btq_int8_matmul(dev(a), dev(sa), dev(w), dev(sw), bf16=False)
        assert_product(y, a, sa, w, sw)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 8, 64, 200])
def test_int8_matmul_nan_and_inf_scales_stay_in_their_rows(T):
    say(f"case: int8_matmul NaN and Inf scales T={T}")
    rng = gen(T)
    a, sa, w, sw, _ = case(rng, 2, T, 96, 256)
    sa[0, T // 2] = np.nan
    sw[1, 5] = np.inf
    sw[1, 95] = np.nan
    y = B.btq_int8_matmul(dev(a), dev(sa), dev(w), dev(sw))
    assert_product(y, a, sa, w, sw)
    got = f32(y)
    assert np.isnan(got[0, T // 2]).all() and np.isfinite(np.delete(got[0], T // 2, 0)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("K", [64, 100, 512])
@pytest.mark.parametrize("T", [1, 20, 150])
def test_int8_matmul_strides_and_alignment(T, K):
    say(f"case: int8_matmul strides T={T} K={K}")
    P, N = 3, 70
    rng = gen(K + T)
    a, sa, w, sw, _ = case(rng, P, T, N, K)
    dw, dsw, dsa = dev(w), dev(sw), dev(sa)
    cols = dev(np.ascontiguousarray(a.transpose(1, 0, 2).reshape(T, P * K)))
    y = B.btq_int8_matmul(cols.view(T, P, K).transpose(0, 1), dsa, dw, dsw)   # column slices
    assert_product(y, a, sa, w, sw, what="column slices")
    for off in (1, 2, 4, 8, 16):       # activations and weights off every vector boundary
        wide = torch.zeros((P, T, K + 32), dtype=torch.int8, device=DEV)
        wide[:, :, off:off + K] = dev(a)
        buf = torch.zeros(P * N * K + 32, dtype=torch.int8, device=DEV)
        wv = buf[off:off + P * N * K].view(P, N, K)
        wv.copy_(dw)
        out = torch.full((P * T * N + 32,), 77.0, device=DEV)
        yv = out[off:off + P * T * N].view(P, T, N)
        y = B.btq_int8_matmul(wide[:, :, off:off + K], dsa, wv, dsw, y=yv)
        assert_product(y, a, sa, w, sw, what=f"offset {off}")
        assert (out[:off] == 77).all() and (out[off + P * T * N:] == 77).all()
        out = torch.full((P * T * N + 32,), 77.0, device=DEV, dtype=torch.bfloat16)
        yv = out[off:off + P * T * N].view(P, T, N)
        y = B.btq_int8_matmul(dev(a), dsa, dw, dsw, y=yv)
        assert_product(y, a, sa, w, sw, what=f"bf16 y, offset {off}")
        assert (out[:off] == 77).all() and (out[off + P * T * N:] == 77).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,N,K", [(140000, 16384, 64), (9, 24, 0)])
def test_int8_matmul_offsets_past_32_bits(T, N, K):
    # y passes 2^31 elements; or the rows of a lie more than 2^32 bytes apart
    say(f"case: int8_matmul offsets past 32 bits T={T} N={N}")
    rng = gen(T)
    if K:
        a, sa, w, sw, _ = case(rng, 1, T, N, K)
        y = B.btq_int8_matmul(dev(a), dev(sa), dev(w), dev(sw))
        rows = np.r_[0:3, T // 2:T // 2 + 3, T - 300:T]
        assert_product(y[:, torch.from_numpy(rows).to(DEV)], a[:, rows], sa[:, rows], w, sw)
    else:
        K, pitch = 256, (1 << 30) + 16
        a, sa, w, sw, _ = case(rng, 1, T, N, K)
        buf = torch.empty(pitch * (T - 1) + K, dtype=torch.int8, device=DEV)
        av = buf.as_strided((1, T, K), (0, pitch, 1))
        av.copy_(dev(a))
        assert_product(B.btq_int8_matmul(av, dev(sa), dev(w), dev(sw)), a, sa, w, sw)


# ---- int8_linear -------------------------------------------------------------

@pytest.mark.gpu
@pytest.mark.parametrize("P,T,N,K", [(1, 1, 8, 5), (8, 1, 512, 1024), (2, 1, 40, 8208), (2, 3, 64, 256),
                                     (2, 8, 320, 512), (3, 16, 48, 100), (1, 40, 96, 2048),
                                     (2, 64, 128, 1008), (3, 77, 99, 1000), (2, 300, 256, 512),
                                     (1, 9, 70, 4096), (2, 5, 33, 8192), (1, 3, 40, 5598),
                                     (2, 33, 40, 2046), (1, 17, 64, 18), (8, 300, 512, 640),
                                     (2, 4, 40, 8194)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_int8_linear_is_the_two_calls(P, T, N, K, dtype):
    say(f"case: int8_linear P={P} T={T} N={N} K={K} {dtype}")
    rng = gen(K + T)
    _, _, w, sw, b = case(rng, P, 1, N, K, bias=True)
    x = torch.randn((P, T, K), device=DEV).to(dtype)
    if T > 2:
        x[0, 1] = 0
        x[P - 1, 2, K - 1] = float("nan")
    dw, dsw, db = dev(w), dev(sw), dev(b)
    for bias in (None, db):
        for bf16 in (True, False):
            y = B.btq_int8_linear(x, dw, dsw, bias=bias, bf16=bf16)
            q, s = B.btq_quantize_rows(x)
            z = B.btq_int8_matmul(q, s, dw, dsw, bias=bias, bf16=bf16)
            assert np.array_equal(f32(y), f32(z), equal_nan=True)
    if dtype == torch.bfloat16:
        codes, scale, _ = codes64(f32(x).astype(np.float64))
        assert_product(B.btq_int8_linear(x, dw, dsw), codes, scale, w, sw)
        assert B.btq_int8_linear(x, dw, dsw).dtype == torch.bfloat16
        assert B.btq_int8_linear(x.view(torch.int16), dw, dsw).dtype == torch.int16
    # the same rows for every shard, by shape and by a zero stride
    y = B.btq_int8_linear(x[0], dw, dsw, bf16=False)
    z = B.btq_int8_linear(x[:1].expand(P, T, K), dw, dsw, bf16=False)
    v = B.btq_int8_linear(x[:1].repeat(P, 1, 1), dw, dsw, bf16=False)
    assert np.array_equal(f32(y), f32(z), equal_nan=True)
    assert np.array_equal(f32(y), f32(v), equal_nan=True)
    # shards as column slices of one matrix
    cols = x.transpose(0, 1).contiguous().transpose(0, 1)
    assert np.array_equal(f32(B.btq_int8_linear(cols, dw, dsw, bf16=False)),
                          f32(B.btq_int8_linear(x, dw, dsw, bf16=False)), equal_nan=True)


@pytest.mark.gpu
def test_int8_linear_approximates_the_bf16_layer():
    # 8-bit codes of both operands: each product's relative error has a
    # standard deviation of about (step/sqrt(12))/rms for either side. With
    # normal rows of 2048 the largest value is below 4.8 sigma, so a step is
    # at most 4.8/127 sigma and the sum's relative error has a deviation below
    # sqrt(2)*4.8/127/sqrt(12) = 1.55%; the check allows 2%.
    say("case: int8_linear against the product in 64 bits of unquantized values")
    P, T, N, K = 2, 64, 256, 2048
    x = torch.randn((P, T, K), device=DEV).to(torch.bfloat16)
    wf = torch.randn((P, N, K), device=DEV)
    w, sw = B.btq_quantize_rows(wf)
    y = f32(B.btq_int8_linear(x, w, sw)).astype(np.float64)
    ex = np.matmul(f32(x).astype(np.float64), wf.cpu().numpy().astype(np.float64).swapaxes(1, 2))
    assert np.linalg.norm(y - ex) <= 0.02 * np.linalg.norm(ex)


@pytest.mark.gpu
def test_empty_batch():
    say("case: empty batches of the 8-bit calls")
    w, sw = torch.ones((2, 8, 16), dtype=torch.int8, device=DEV), torch.ones((2, 8), device=DEV)
    x = torch.empty((2, 0, 16), device=DEV)
    assert B.btq_int8_linear(x, w, sw).shape == (2, 0, 8)
    q, s = B.btq_quantize_rows(x)
    assert q.shape == (2, 0, 16) and s.shape == (2, 0)
    assert B.btq_int8_matmul(q, s, w, sw).shape == (2, 0, 8)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 24, 300])
def test_int8_linear_side_stream_and_graph(T):
    say(f"case: int8_linear on a side stream and in a graph T={T}")
    P, N, K = 2, 160, 512
    w, sw = B.btq_quantize_rows(torch.randn((P, N, K), device=DEV))
    xs = [torch.randn((P, T, K), device=DEV).to(torch.bfloat16) for _ in range(4)]
    ref = [B.btq_int8_linear(x, w, sw) for x in xs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream(device=DEV)   # default priority
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)      # a bounded spin: the side stream runs late
    got = [B.btq_int8_linear(x, w, sw, stream=side) for x in xs]
    junk = [torch.full((1 << 18,), -7, dtype=torch.int32, device=DEV) for _ in range(16)]
    side.synchronize()
    torch.cuda.synchronize()
    del junk
    for a, b in zip(ref, got):
        assert torch.equal(a, b)
    x, y = xs[0].clone(), torch.empty_like(ref[0])
    ws = torch.empty(B.btq_int8_linear_workspace_bytes(P, T, K), dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.btq_int8_linear(x, w, sw, y=y, workspace=ws)
    for xi, r in zip(xs, ref):
        x.copy_(xi)
        ws.fill_(0x5A)
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, r)


# ---- refusals (CPU): all return before any HIP call ----------------------------

A, BIG = 0x10000, 1 << 40
OK, ARG, SHAPE, ALIGN, WS = (_lib.BTQ_OK, _lib.BTQ_ERR_ARG, _lib.BTQ_ERR_SHAPE,
                             _lib.BTQ_ERR_ALIGN, _lib.BTQ_ERR_WORKSPACE)


def test_quantize_rows_refusals():
    lib = _lib.load()

    def call(x=A, xt=1, sh=64, pi=16, P=1, T=4, K=16, q=A, s=A):
        return lib.btq_quantize_rows(x, xt, sh, pi, P, T, K, q, s, None)
    for kw in (dict(P=0), dict(K=0), dict(T=-1), dict(P=70000), dict(K=(1 << 30) + 1),
               dict(sh=-1), dict(pi=-1), dict(pi=1 << 61), dict(T=1 << 50, K=1 << 20)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(x=None), dict(q=None), dict(s=None), dict(xt=2), dict(xt=-1)):
        assert call(**kw) == ARG, kw
    for kw in (dict(x=A + 1), dict(x=A + 2, xt=0), dict(s=A + 2)):
        assert call(**kw) == ALIGN, kw
    assert call(T=0, x=None, q=None, s=None) == OK


def test_int8_matmul_refusals():
    lib = _lib.load()

    def call(a=A, ash=64, ap=16, sa=A, ssh=4, w=A, sw=A, b=None, P=1, T=4, N=8, K=16, y=A, yt=1):
        return lib.btq_int8_matmul(a, ash, ap, sa, ssh, w, sw, b, P, T, N, K, y, yt, None)
    for kw in (dict(P=0), dict(N=0), dict(K=0), dict(T=-1), dict(K=131072), dict(ash=-1),
               dict(ap=-1), dict(ssh=-1), dict(N=(1 << 30) + 1), dict(P=70000),
               dict(T=1 << 50, N=1 << 20), dict(ap=1 << 61)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(a=None), dict(sa=None), dict(w=None), dict(sw=None), dict(y=None), dict(yt=2),
               dict(yt=7)):
        assert call(**kw) == ARG, kw
    for kw in (dict(sa=A + 1), dict(sw=A + 2), dict(b=A + 2), dict(y=A + 1), dict(y=A + 2, yt=0)):
        assert call(**kw) == ALIGN, kw
    assert call(T=0, a=None, sa=None, y=None) == OK


def test_int8_linear_refusals():
    lib = _lib.load()

    def call(x=A, xt=1, sh=64, pi=16, w=A, sw=A, b=None, P=1, T=4, N=8, K=16, y=A, yt=1, ws=A,
             wsb=BIG):
        return lib.btq_int8_linear(x, xt, sh, pi, w, sw, b, P, T, N, K, y, yt, ws, wsb, None)
    for kw in (dict(P=0), dict(N=0), dict(K=131072), dict(T=-1), dict(sh=-1), dict(pi=-1)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(x=None), dict(w=None), dict(sw=None), dict(y=None), dict(ws=None), dict(xt=2),
               dict(yt=2)):
        assert call(**kw) == ARG, kw
    for kw in (dict(x=A + 1), dict(ws=A + 8), dict(y=A + 1), dict(b=A + 1)):
        assert call(**kw) == ALIGN, kw
    need = lib.btq_int8_linear_workspace_bytes(2, 4, 17)
    assert need >= 2 * 4 * (17 + 4)
    assert call(P=2, K=17, wsb=need - 1) == WS
    for bad in ((0, 4, 16), (1, -1, 16), (1, 4, 0), (1, 4, 131072)):
        assert lib.btq_int8_linear_workspace_bytes(*bad) == 0
    assert call(T=0, x=None, y=None, ws=None, wsb=0) == OK


def test_binding_refuses_host_tensors():
    x = torch.zeros((2, 4, 16), dtype=torch.bfloat16)
    w, sw = torch.zeros((2, 8, 16), dtype=torch.int8), torch.zeros((2, 8))
    with pytest.raises(ValueError):
        B.btq_quantize_rows(x)
    with pytest.raises(ValueError):
        B.btq_int8_linear(x, w, sw)
    with pytest.raises(ValueError):
        B.btq_int8_matmul(x.to(torch.int8), sw, w, sw)


@pytest.mark.gpu
def test_binding_refusals():
    say("case: the 8-bit binding's argument checks")
    x = torch.zeros((2, 4, 16), dtype=torch.bfloat16, device=DEV)
    w, sw = torch.zeros((2, 8, 16), dtype=torch.int8, device=DEV), torch.zeros((2, 8), device=DEV)
    q, s = B.btq_quantize_rows(x)
    for exc, call in (
            (TypeError, lambda: B.btq_quantize_rows(x.double())),
            (ValueError, lambda: B.btq_quantize_rows(x[0, 0])),
            (ValueError, lambda: B.btq_quantize_rows(x.transpose(1, 2))),
            (ValueError, lambda: B.btq_quantize_rows(x, q=q[:1])),
            (TypeError, lambda: B.btq_quantize_rows(x, q=q.float())),
            (TypeError, lambda: B.btq_int8_matmul(x, s, w, sw)),
            (ValueError, lambda: B.btq_int8_matmul(q, s, w[:, :, :8], sw)),
            (ValueError, lambda: B.btq_int8_matmul(q, s, w[:1], sw)),
            (ValueError, lambda: B.btq_int8_matmul(q, s[:1], w, sw)),
            (ValueError, lambda: B.btq_int8_matmul(q, s, w, sw[:, :4])),
            (ValueError, lambda: B.btq_int8_matmul(q, s, w, sw, bias=sw[0])),
            (TypeError, lambda: B.btq_int8_matmul(q, s, w.float(), sw)),
            (TypeError, lambda: B.btq_int8_matmul(q, s, w, sw, y=q)),
            (ValueError, lambda: B.btq_int8_matmul(q, s, w, sw, y=sw)),
            (ValueError, lambda: B.btq_int8_matmul(q, s.cpu(), w, sw)),
            (RuntimeError, lambda: B.btq_int8_linear(x, w, sw, workspace=q.view(-1)[:16])),
            (TypeError, lambda: B.btq_int8_linear(q, w, sw))):
        with pytest.raises(exc):
            call()
