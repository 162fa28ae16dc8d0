"""btq_kv_append and btq_kv_gather: the cache's bytes and the gathered values bit for
bit against numpy, which takes the fp32 steps that the header names."""
import numpy as np
import pytest
import torch

import bit_tensor_activation_amd as B
from bit_tensor_activation_amd import _lib
from helpers import say
from kv_helpers import (BF16, DEV, F32, Batch, block_bytes, host32, put, quantize, table, turn,
                        unpack)


def rounded(x, dtype):
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


def same(a, b):
    """Equal bits, NaNs equal."""
    a, b = a.float().cpu(), b.float().cpu()
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


def expect(batch, cache, k, v, cos, sin, style):
    """What the cache (numpy, changed in place) holds after the append, and the
    gathered keys and values in fp32."""
    P, T, Hk, D = k.shape
    ko, vo = np.zeros(k.shape, np.float32), np.zeros(v.shape, np.float32)
    for row, b, place in batch.rows():
        x, y = k[:, row], v[:, row]
        if cos is not None and place >= 0:
            if place < len(cos):
                with np.errstate(invalid="ignore", over="ignore"):
                    x = turn(x, cos[place], sin[place], style)
            else:
                x = x.copy()
                x[..., :2 * cos.shape[-1]] = np.nan
        at = batch.where(b, place)
        if at is None:
            continue
        for out, src, key in ((ko, x, True), (vo, y, False)):
            c, s, z, w = quantize(src)
            for p in range(P):
                for h in range(Hk):
                    pair = (c[p, h], w[p, h])
                    put(cache, at, p, h, D, **({"k": pair} if key else {"v": pair}))
            s = np.where((w >> 16) == 0x7fc0, np.nan, s).astype(np.float32)
            out[:, row] = (c - z[..., None]).astype(np.float32) * s[..., None]
    return ko, vo


def check(batch, P, Hk, D, dim=0, style="half", dt=BF16, make=None, rows=None, fused=True, y_dt=F32,
          shift=0):
    g = np.random.default_rng(batch.T * 31 + D + Hk)
    T = batch.T
    x = g.standard_normal((P, T, 3 * Hk, D)).astype(np.float32)
    x[..., :1] *= 5
    if make is not None:
        make(x[:, :, :Hk], x[:, :, Hk:2 * Hk])
    buf = torch.zeros(x.size + shift, dtype=dt, device=DEV)
    buf[shift:] = torch.from_numpy(x.reshape(-1)).to(DEV).to(dt)
    x = buf[shift:].view(P, T, 3 * Hk, D)
    k, v = x[:, :, :Hk], x[:, :, Hk:2 * Hk]
    if not fused:
        k, v = k.contiguous(), v.contiguous()
    cos = sin = c = s = None
    if dim:
        cos, sin = table(rows or max(batch.lengths + [1]), dim)
        c, s = host32(cos), host32(sin)
    shape = (P, batch.pages, Hk, batch.page // 32, block_bytes(D))
    before = g.integers(0, 256, shape, dtype=np.uint8)
    cache = torch.from_numpy(before.copy()).to(DEV)
    starts, lengths, tb = batch.dev()
    B.btq_kv_append(k, v, starts, lengths, tb, cache, cos=cos, sin=sin, rope=style)
    want = before.copy()
    ko, vo = expect(batch, want, host32(k), host32(v), c, s, style)
    got = cache.cpu().numpy()
    wrong = np.argwhere(got != want)
    assert len(wrong) == 0, f"{len(wrong)} bytes differ, first at {wrong[0]}"

    ko, vo = rounded(ko, y_dt), rounded(vo, y_dt)
    full = torch.full((2, P, T, Hk, D), 7.0, dtype=y_dt, device=DEV)
    gk, gv = B.btq_kv_gather(starts, lengths, tb, cache, k=full[0], v=full[1])
    own = np.zeros(T, bool)
    for row, _, _ in batch.rows():
        own[row] = True
    assert same(gk[:, own], ko[:, own]) and same(gv[:, own], vo[:, own])
    assert (gk[:, ~own] == 7).all() and (gv[:, ~own] == 7).all()
    return cache


BATCHES = [
    Batch([1], [1]), Batch([1], [32]), Batch([1], [33]), Batch([33], [33]), Batch([32], [64]),
    Batch([1] * 9, [1, 2, 31, 32, 33, 63, 64, 65, 100]),
    Batch([5, 0, 70, 1], [5, 12, 93, 64], page=64, before=3, behind=4),
    Batch([7, 40, 3], [200, 41, 3], page=128, slack=2),
    Batch([0, 0], [0, 40]), Batch([64, 64, 64], [64, 65, 79]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("n", range(len(BATCHES)))
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
def test_batches(n, D):
    say(f"case: kv append batch {n} D={D}")
    check(BATCHES[n], 2, 1, D, dim=D)
    check(BATCHES[n], 1, 3, D, dim=D // 2, style="pairs", y_dt=BF16)


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF16, F32])
@pytest.mark.parametrize("dim", [0, 2, 10, 48, 64, 126, 128])
def test_rotations_and_types(dt, dim):
    for style in ("half", "pairs"):
        check(BATCHES[6], 2, 2, 128, dim=dim, style=style, dt=dt, fused=False)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
def test_part_of_a_head_turned(D):
    say(f"case: kv append part turned D={D}")
    for style in ("half", "pairs"):
        for dim in {D // 4, D // 2, 3 * D // 4, min(D, 64)}:
            check(BATCHES[6], 1, 2, D, dim=dim, style=style, dt=BF16, fused=False)
            check(BATCHES[7], 1, 1, D, dim=dim, style=style, dt=F32, fused=False)


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [0, 1, 2, 3, 4, 8])
def test_rows_on_any_element(shift):
    for dt in (BF16, F32):
        check(BATCHES[7], 2, 2, 64, dim=32, dt=dt, shift=shift)


@pytest.mark.gpu
def test_special_rows():
    # zeros, a constant of each sign, NaN, Inf, ties of every code, tiny and huge ranges
    def make(k, v):
        for x in (k, v):
            x[:, 0] = 0
            x[:, 1] = 2.5
            x[:, 2] = -2.5
            x[:, 3, :, 7] = np.nan
            x[:, 4, :, 0] = np.inf
            x[:, 5, :, 63] = -np.inf
            x[:, 6] = np.tile(np.arange(64) / 2 - 7.5, 1)[:64].clip(-7.5, 7.5)
            x[:, 7] = (np.arange(64) % 31) / 2
            x[:, 8] *= 1e-39
            x[:, 9] *= 1e-37
            x[:, 10] *= 1e38
            x[:, 10, :, :2] = [3e38, -3e38]
            x[:, 11, :, :2] = [1.5e38, -1.5e38]
            x[:, 12] = 0
            x[:, 12, :, 5] = 1e-45
    b = Batch([14, 13], [40, 13])
    for dt in (BF16, F32):
        check(b, 2, 2, 64, dt=dt, make=make)
        check(b, 1, 2, 64, dt=dt, make=make, dim=64)


@pytest.mark.gpu
def test_error_of_a_code_is_half_a_step():
    b = Batch([500], [500])
    cache = check(b, 1, 1, 128, fused=False)
    k, v = unpack(cache.cpu().numpy(), 128)
    assert np.isfinite(k[:, b.table[0]]).all() and np.isfinite(v[:, b.table[0]][:, :15]).all()


@pytest.mark.gpu
def test_places_without_a_page_and_before_the_sequence():
    b = Batch([50, 20, 10], [100, 12, 10], page=32)   # 8 rows of the second have no place
    b.table[0, 2] = -1
    b.table[2, 0] = b.pages
    check(b, 2, 1, 64, dim=64)
    b = Batch([10, 90], [10, 90])
    b.max_pages = 2                                     # the table is shorter than a sequence
    b.table = np.ascontiguousarray(b.table[:, :2])
    b.lengths[1] = 64                                   # (what lengths are cut to)
    starts, lengths, tb = b.dev()
    b.lengths[1] = 64
    check(b, 1, 1, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("D,dim", [(128, 128), (128, 10), (192, 64)])
def test_rows_before_the_sequence_with_tables(D, dim):
    # far more rows than places: the others' places are negative, and their rows of the
    # tables are none (nothing before the tables is read)
    b = Batch([700, 90], [12, 40], page=32)
    check(b, 1, 2, D, dim=dim)
    check(b, 1, 1, D, dim=dim, style="pairs", dt=F32, rows=5)


@pytest.mark.gpu
def test_positions_past_the_table_are_nan():
    check(Batch([6], [40]), 1, 1, 64, dim=32, rows=37)


@pytest.mark.gpu
def test_long_cache_offsets_pass_32_bits():
    # 6 GB of pages; the ones in use lie at the end and at both sides of 4 GiB
    D, page = 128, 64
    per = page // 32 * block_bytes(D)
    pages = (6 << 30) // per
    cache = torch.zeros((1, pages, 1, page // 32, block_bytes(D)), dtype=torch.uint8, device=DEV)
    b = Batch([150], [170], page=page)
    b.table[0, :3] = [pages - 1, (4 << 30) // per, (4 << 30) // per - 1]
    b.pages = pages
    x = torch.randn((1, 150, 2, D), device=DEV).to(BF16)
    starts, lengths, tb = b.dev()
    B.btq_kv_append(x[:, :, :1], x[:, :, 1:], starts, lengths, tb, cache)
    k, v = B.btq_kv_gather(starts, lengths, tb, cache, tokens=150, dtype=F32)
    for got, src in ((k, x[:, :, :1]), (v, x[:, :, 1:])):
        c, s, z, _ = quantize(host32(src))
        assert same(got, torch.from_numpy((c - z[..., None]).astype(np.float32) * s[..., None]))
    small = torch.zeros_like(cache[:, :3])
    b.table[0, :3] = [0, 1, 2]
    B.btq_kv_append(x[:, :, :1], x[:, :, 1:], starts, lengths, torch.from_numpy(b.table).to(DEV), small)
    for i, p in enumerate((pages - 1, (4 << 30) // per, (4 << 30) // per - 1)):
        assert torch.equal(cache[0, p], small[0, i])


@pytest.mark.gpu
def test_pieces_give_the_bytes_of_the_whole():
    # a prompt in one call, and in pieces that end inside bytes, blocks and pages
    T, D = 203, 128
    x = torch.randn((2, T, 2, D), device=DEV).to(BF16)
    k, v = x[:, :, :1], x[:, :, 1:]
    cos, sin = table(T, D)
    whole = Batch([T], [T], page=64)
    tb = torch.from_numpy(whole.table).to(DEV)
    a = torch.zeros((2, whole.pages, 1, 2, block_bytes(D)), dtype=torch.uint8, device=DEV)
    b = torch.zeros_like(a)
    starts, lengths, _ = whole.dev()
    B.btq_kv_append(k, v, starts, lengths, tb, a, cos=cos, sin=sin)
    at = 0
    for n in (1, 1, 30, 1, 64, 5, 27, 62, 12):
        st = torch.tensor([0, n], dtype=torch.int32, device=DEV)
        ln = torch.tensor([at + n], dtype=torch.int32, device=DEV)
        B.btq_kv_append(k[:, at:at + n], v[:, at:at + n], st, ln, tb, b, cos=cos, sin=sin)
        at += n
    assert at == T and torch.equal(a, b)


@pytest.mark.gpu
def test_gather_of_one_and_of_any_stretch():
    b = Batch([90, 40], [90, 40])
    cache = check(b, 2, 2, 64, dim=64)
    starts, lengths, tb = b.dev()
    k, v = B.btq_kv_gather(starts, lengths, tb, cache, tokens=130)
    only = torch.empty_like(v)
    assert B.btq_kv_gather(starts, lengths, tb, cache, v=only)[0] is None
    assert torch.equal(only, v)
    st = torch.tensor([0, 30, 35], dtype=torch.int32, device=DEV)
    ln = torch.tensor([57, 20], dtype=torch.int32, device=DEV)
    k2, v2 = B.btq_kv_gather(st, ln, tb, cache, tokens=37)
    assert torch.equal(k2[:, :30], k[:, 27:57]) and torch.equal(v2[:, 30:35], v[:, 105:110])
    assert (k2[:, 35:] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("first,last", [(-5, 4), (-2 ** 31, 0), (0, 3), (-40, 2 ** 31 - 11 - 70)])
def test_starts_outside_the_batch_are_cut(first, last):
    # the same bytes and rows as with starts cut to [0,T]
    b = Batch([40, 30, 5], [90, 30, 5], page=32)
    starts, lengths, tb = b.dev()
    x = torch.randn((2, b.T, 2, 64), device=DEV).to(BF16)
    wide = starts.clone()
    wide[0] = first
    wide[-1] += last
    held = []
    for st in (starts, wide):
        cache = torch.zeros((2, b.pages, 1, 1, block_bytes(64)), dtype=torch.uint8, device=DEV)
        B.btq_kv_append(x[:, :, :1], x[:, :, 1:], st, lengths, tb, cache)
        held.append((cache, *B.btq_kv_gather(st, lengths, tb, cache, tokens=b.T)))
    for got, want in zip(held[1], held[0]):
        assert want.any() and torch.equal(got, want)


@pytest.mark.gpu
def test_no_shards_and_empty_batches():
    b = Batch([40], [40])
    x = torch.randn((40, 4, 64), device=DEV).to(BF16)
    starts, lengths, tb = b.dev()
    c3 = torch.zeros((b.pages, 2, 1, block_bytes(64)), dtype=torch.uint8, device=DEV)
    c4 = torch.zeros_like(c3)[None]
    B.btq_kv_append(x[:, :2], x[:, 2:], starts, lengths, tb, c3)
    B.btq_kv_append(x[None, :, :2], x[None, :, 2:], starts, lengths, tb, c4)
    assert torch.equal(c3, c4[0]) and c3.any()
    k, v = B.btq_kv_gather(starts, lengths, tb, c3, tokens=40)
    assert k.shape == v.shape == (40, 2, 64)
    none = torch.zeros((1,), dtype=torch.int32, device=DEV)
    e = torch.empty((0, 2, 64), dtype=BF16, device=DEV)
    B.btq_kv_append(e, e, none, none[:0], tb[:0], c3)
    B.btq_kv_append(x[:, :2], x[:, 2:], none, none[:0], tb[:0], c3)
    assert torch.equal(c3, c4[0])


@pytest.mark.gpu
def test_python_refusals():
    b = Batch([4], [4])
    starts, lengths, tb = b.dev()
    x = torch.zeros((1, 4, 2, 64), dtype=BF16, device=DEV)
    cache = torch.zeros((1, b.pages, 2, 1, block_bytes(64)), dtype=torch.uint8, device=DEV)
    args = dict(k=x, v=x, seq_starts=starts, lengths=lengths, page_table=tb, cache=cache)
    for kw in (dict(v=x[:, :3]), dict(cache=cache[0]), dict(seq_starts=starts[:1]),
               dict(page_table=tb[0]), dict(rope="x"), dict(cos=table(4, 64)[0]),
               dict(k=x[:, :, :1], v=x[:, :, :1]), dict(k=x[0], v=x[0]),
               dict(cache=torch.cat((cache, cache))), dict(v=x[..., ::2])):
        with pytest.raises(ValueError):
            B.btq_kv_append(**{**args, **kw})
    for kw in (dict(v=x.float()), dict(lengths=lengths.long()), dict(cache=cache.char()),
               dict(k=x.half(), v=x.half())):
        with pytest.raises(TypeError):
            B.btq_kv_append(**{**args, **kw})
    with pytest.raises(ValueError):
        B.btq_kv_gather(starts, lengths, tb, cache)
    with pytest.raises(ValueError):
        B.btq_kv_gather(starts, lengths, tb, cache, k=x[0])
    three = torch.zeros((1, 1, 2, 3, block_bytes(64)), dtype=torch.uint8, device=DEV)
    with pytest.raises(RuntimeError):
        B.btq_kv_append(**{**args, "cache": three})


# ---- CPU: all return before any HIP call ---------------------------------------

A = 0x10000
OK, ARG, SHAPE, ALIGN = _lib.BTQ_OK, _lib.BTQ_ERR_ARG, _lib.BTQ_ERR_SHAPE, _lib.BTQ_ERR_ALIGN


def test_block_bytes():
    f = _lib.load().btq_kv_block_bytes
    assert [f(d) for d in (32, 64, 96, 128, 256)] == [1280, 2304, 3328, 4352, 8448]
    assert [f(d) for d in (0, -32, 16, 33, 80, 288, 1 << 40)] == [0] * 7
    assert B.btq_kv_block_bytes(128) == 4352
    with pytest.raises(ValueError):
        B.btq_kv_block_bytes(100)


def append(k=A, v=A, xt=1, ks=0, kp=256, kh=128, vs=0, vp=256, vh=128, P=1, T=4, Hk=2, D=128,
           starts=A, lengths=A, nb=1, tb=A, mp=2, cos=A, sin=A, rows=16, dim=128, rope=0, cache=A,
           pages=4, size=64):
    return _lib.load().btq_kv_append(k, v, xt, ks, kp, kh, vs, vp, vh, P, T, Hk, D, starts,
                                     lengths, nb, tb, mp, cos, sin, rows, dim, rope, cache, pages,
                                     size, None)


def gather(starts=A, lengths=A, nb=1, tb=A, mp=2, cache=A, pages=4, size=64, P=1, T=4, Hk=2, D=128,
           k=A, v=A, yt=1, ks=0, kp=256, kh=128, vs=0, vp=256, vh=128):
    return _lib.load().btq_kv_gather(starts, lengths, nb, tb, mp, cache, pages, size, P, T, Hk, D,
                                     k, v, yt, ks, kp, kh, vs, vp, vh, None)


SHAPES = [dict(P=0), dict(P=65536), dict(T=-1), dict(T=(1 << 30) + 1), dict(Hk=0), dict(Hk=65536),
          dict(D=16), dict(D=80), dict(D=288), dict(nb=-1), dict(nb=(1 << 30) + 1), dict(mp=-1),
          dict(size=16), dict(size=48), dict(size=0), dict(size=-64), dict(size=1 << 17),
          dict(mp=(1 << 24) + 1), dict(pages=0), dict(pages=1 << 31), dict(pages=1 << 60),
          dict(P=65535, Hk=200), dict(T=1 << 30, P=8), dict(ks=-1, P=2), dict(kp=-1), dict(vh=-1),
          dict(kp=1 << 61), dict(P=2, vs=1 << 61)]


def test_append_refusals():
    assert append(T=0) == OK and append(nb=0) == OK
    for kw in SHAPES + [dict(dim=0), dict(dim=5), dict(dim=130), dict(rows=0)]:
        assert append(**kw) == SHAPE, kw
    for kw in (dict(k=None), dict(v=None), dict(xt=2), dict(starts=None), dict(lengths=None),
               dict(tb=None), dict(cache=None), dict(cos=None), dict(sin=None), dict(rope=2)):
        assert append(**kw) == ARG, kw
    for kw in (dict(k=A + 1), dict(v=A + 1), dict(xt=0, v=A + 2), dict(starts=A + 2),
               dict(lengths=A + 1), dict(tb=A + 2), dict(cache=A + 8), dict(cos=A + 2)):
        assert append(**kw) == ALIGN, kw


def test_gather_refusals():
    assert gather(T=0) == OK and gather(nb=0) == OK
    for kw in SHAPES:
        assert gather(**kw) == SHAPE, kw
    for kw in (dict(k=None, v=None), dict(yt=2), dict(starts=None), dict(lengths=None),
               dict(tb=None), dict(cache=None)):
        assert gather(**kw) == ARG, kw
    for kw in (dict(k=A + 1), dict(v=A + 1), dict(yt=0, v=A + 2), dict(cache=A + 4)):
        assert gather(**kw) == ALIGN, kw


def test_gather_into_overlapping_heads():
    for kw in (dict(kh=0), dict(kp=0), dict(vh=127), dict(vp=255), dict(P=2, ks=0, vs=1024),
               dict(P=2, ks=1024, vs=0)):
        assert gather(**kw) == SHAPE, kw
        assert append(**kw, k=None) == ARG, kw          # the same strides of inputs
    assert gather(k=None, v=None, kh=0, vh=0) == ARG
    assert gather(k=None, ks=0, kp=0, kh=0, v=A + 1) == ALIGN    # (one that is not written)
    assert gather(T=1, kp=0, vp=0, k=A + 1) == ALIGN
