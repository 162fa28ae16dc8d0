"""btq_kv_attention against plain numpy in 64 bits (kv_helpers.attention, which
derives the tolerance; the output's own rounding and a factor 1.05 for terms of
second order are added here)."""
import numpy as np
import pytest
import torch

import bit_tensor_activation_amd as B
from bit_tensor_activation_amd import _lib
from helpers import say
from kv_helpers import (BF16, DEV, F32, NAN_WORD, U, Batch, attention, block_bytes, host,
                        random_cache)


def compare(got, lse, want, dt):
    out, tol, l, ltol = want
    P, T, Hq, D = out.shape
    got, own = host(got).reshape(P, T, Hq, D), ~np.isnan(out)
    tol = 1.05 * tol + (U if dt == F32 else 2.0 ** -8) * np.abs(out) + 2.0 ** -133
    off = np.abs(got - out)
    assert (off[own] <= tol[own]).all(), (
        f"{(off > tol)[own].sum()} of {own.sum()} off, worst {np.max((off - tol)[own])} at "
        f"{np.argwhere((off > tol) & own)[:3]}, NaN {np.isnan(got[own]).sum()}")
    if lse is not None:
        lse, own = host(lse), ~np.isnan(l)
        none = own & np.isneginf(l)
        assert (lse[none] == -np.inf).all()
        own &= ~none
        assert (np.abs(lse - l)[own] <= (1.05 * ltol)[own]).all(), np.max((np.abs(lse - l) - ltol)[own])


def check(batch, P, Hq, Hk, D, causal=True, window=0, dt=BF16, lse=True, max_length=0, seed=0,
          sigma=1.0, q_sigma=1.5, edit=None, gap=0, shift=0, scale=None):
    g = np.random.default_rng(seed + batch.T + 7 * D)
    size = P * batch.T * (Hq * D + gap) + shift
    flat = torch.from_numpy((g.standard_normal(size) * q_sigma).astype(np.float32)).to(DEV).to(BF16)
    q = flat[shift:].view(P, batch.T, Hq * D + gap)[..., :Hq * D].unflatten(-1, (Hq, D))
    cache = random_cache(batch, P, Hk, D, seed, sigma)
    if edit is not None:
        edit(batch, cache)
    starts, lengths, tb = batch.dev()
    out = torch.full((P, batch.T, Hq * D), 5.0, dtype=dt, device=DEV)
    sums = torch.full((P, batch.T, Hq), 5.0, device=DEV) if lse else None
    dev = torch.from_numpy(cache).to(DEV)
    got = B.btq_kv_attention(q, starts, lengths, tb, dev, causal=causal, window=window,
                             max_length=max_length, out=out, lse=sums, scale=scale)
    assert got is out
    want = attention(batch, cache, host(q), Hk, D, D ** -0.5 if scale is None else float(np.float32(scale)),
                     causal, window)
    compare(out, sums, want, dt)
    own = np.zeros(batch.T, bool)
    for row, _, _ in batch.rows():
        own[row] = True
    assert (out[:, ~own] == 5).all()
    assert sums is None or (sums[:, ~own] == 5).all()
    return out, sums, (q, starts, lengths, tb, dev)


BATCHES = [
    Batch([1], [1]), Batch([1], [2]), Batch([1], [31]), Batch([1], [128]), Batch([1], [129]),
    Batch([1], [700], page=64), Batch([1] * 6, [1, 40, 127, 128, 300, 513], page=128),
    Batch([3, 1, 0, 7], [3, 260, 50, 130], before=2, behind=3, slack=1),
    Batch([40, 9], [40, 200], page=64), Batch([0, 2, 0], [0, 2, 9]), Batch([130], [130]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("n", range(len(BATCHES)))
@pytest.mark.parametrize("D", [64, 128])
def test_batches(n, D):
    say(f"case: kv attention batch {n} D={D}")
    check(BATCHES[n], 1, 4, 1, D)
    check(BATCHES[n], 2, 2, 2, D, dt=F32)
    check(BATCHES[n], 1, 6, 2, D, causal=False, lse=False)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [32, 96, 160, 192, 224, 256])
def test_head_sizes(D):
    say(f"case: kv attention D={D}")
    for n in (5, 7, 8):
        check(BATCHES[n], 2, 4, 1, D)
    check(BATCHES[10], 1, 8, 1, D)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 3), (8, 1), (5, 1), (16, 1), (17, 1), (40, 2), (64, 1),
                                   (12, 4)])
def test_head_groups(Hq, Hk):
    say(f"case: kv attention Hq={Hq} Hk={Hk}")
    check(Batch([1, 1], [90, 300]), 1, Hq, Hk, 64)
    check(Batch([5, 2], [90, 150]), 1, Hq, Hk, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 128, 200, 1 << 29, (1 << 31) + 5])
def test_windows(window):
    for causal in (True, False):
        check(BATCHES[7], 1, 4, 1, 64, window=window, causal=causal)
        check(BATCHES[6], 1, 4, 1, 64, window=window, causal=causal)
        check(Batch([70], [300]), 1, 4, 1, 64, window=window, causal=causal)


@pytest.mark.gpu
@pytest.mark.parametrize("length", [512, 513, 2048, 5000])
def test_split_keys(length):
    # one sequence on a whole chip: the keys are split, and by other bounds of length
    # otherwise; rows that stay in one split among them
    say(f"case: kv attention length={length}")
    for ml in (0, length, 128, 1 << 20):
        check(Batch([1], [length], page=64), 1, 8, 1, 128, max_length=ml, dt=F32)
    check(Batch([2, 1, 1], [length, 3, 900], page=64), 1, 4, 2, 64, dt=F32)
    check(Batch([40], [length], page=64), 1, 8, 1, 64, dt=F32)
    check(Batch([40], [length], page=64), 1, 8, 1, 64, dt=F32, window=1000)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160])
def test_few_columns_on_average(D):
    # groups of 8 columns, several of them in some sequences and rows of two in some
    for Hq in (1, 3, 4):
        b = Batch([9, 1, 0, 1, 2, 1, 1, 1, 1, 1, 0, 1, 0], [300, 1, 7, 129, 64, 513, 33, 2, 96, 700, 3, 40, 0], page=64)
        check(b, 2, Hq, 1, D, dt=F32)
        check(b, 1, 2 * Hq, 2, D, window=70, causal=Hq != 3)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
def test_shares_of_long_keys(D):
    # equal shares of the keys, few columns and more than one group of them
    say(f"case: kv attention shares D={D}")
    for b, Hq in ((Batch([1, 2], [4700, 2300], page=64), 2), (Batch([1], [9000], page=64), 5),
                  (Batch([1, 0, 3], [2500, 40, 4100], page=32, before=1, behind=1), 6),
                  (Batch([1], [4200], page=64), 17)):
        check(b, 1, Hq, 1, D, dt=F32)
    check(Batch([1, 2], [4700, 2300], page=64), 1, 4, 1, D, window=3000, causal=D % 64 == 0)


@pytest.mark.gpu
def test_rows_that_see_nothing():
    # more rows than places, no pages, an empty sequence, a table without places
    b = Batch([12, 4, 5], [4, 64, 0])
    b.table[1, :] = -1
    out, lse, _ = check(b, 2, 4, 1, 64)
    assert (out[:, :8] == 0).all() and torch.isneginf(lse[:, :8]).all()
    assert (out[:, 12:] == 0).all()
    b = Batch([3], [3])
    b.table, b.max_pages = np.zeros((1, 0), np.int32), 0
    out, _, _ = check(b, 1, 2, 1, 64)
    assert (out == 0).all()


@pytest.mark.gpu
def test_missing_pages_inside_a_sequence():
    b = Batch([2, 1], [400, 300], page=32)
    b.table[0, [0, 3, 4, 5, 6, 11]] = -1
    b.table[1, 5] = b.pages
    b.table[1, 2] = -2 ** 31
    check(b, 1, 4, 1, 128)
    check(b, 1, 4, 1, 128, window=60)


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["key", "value"])
def test_nan_rows_reach_only_the_queries_that_see_them(what):
    D = 64

    def edit(batch, cache):
        for b, place in ((0, 150), (1, 10)):
            page, block, t = batch.where(b, place)
            at = 32 * D + (128 if what == "value" else 0) + 4 * t
            cache[:, page, :, block, at:at + 4] = np.frombuffer(np.uint32(NAN_WORD).tobytes(), np.uint8)
    b = Batch([60, 1, 1], [180, 400, 30])     # row 30 of the first is place 150
    g = np.random.default_rng(3)
    q = torch.from_numpy(g.standard_normal((1, b.T, 4, D)).astype(np.float32)).to(DEV).to(BF16)
    clean = random_cache(b, 1, 2, D)
    dirty = clean.copy()
    edit(b, dirty)
    starts, lengths, tb = b.dev()
    for kw in (dict(), dict(window=20)):
        a = B.btq_kv_attention(q, starts, lengths, tb, torch.from_numpy(clean).to(DEV), **kw)
        d = B.btq_kv_attention(q, starts, lengths, tb, torch.from_numpy(dirty).to(DEV), **kw)
        sees = torch.zeros(b.T, dtype=torch.bool)
        sees[30:50 if kw else 60] = True
        sees[60] = not kw
        assert torch.isfinite(a).all()
        assert torch.isnan(d[0, sees]).all()
        assert torch.equal(d[0, ~sees], a[0, ~sees])


@pytest.mark.gpu
def test_stale_places_past_the_end_do_not_matter():
    # NaN words, and any bytes, behind the last token and in pages of no sequence
    def edit(batch, cache):
        keep = np.zeros(cache.shape[1:2] + cache.shape[3:4] + (32,), bool)
        for b in range(batch.B):
            for j in range(batch.lengths[b]):
                keep[batch.where(b, j)] = True
        for page, block, t in np.argwhere(~keep):
            for at in (32 * 64 + 4 * t, 32 * 64 + 128 + 4 * t):
                cache[:, page, :, block, at:at + 4] = 0xff
    check(Batch([1, 1, 4], [37, 129, 70], page=64), 2, 4, 1, 64, edit=edit)
    check(Batch([50], [50], page=64), 2, 4, 1, 64, edit=edit)


@pytest.mark.gpu
def test_nan_and_inf_queries_stay_in_their_row():
    b = Batch([1, 1, 40], [300, 300, 60])
    cache = torch.from_numpy(random_cache(b, 1, 1, 128)).to(DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    q = torch.randn((1, b.T, 2, 128), device=DEV, generator=g).to(BF16)
    starts, lengths, tb = b.dev()
    a = B.btq_kv_attention(q, starts, lengths, tb, cache)
    bad = q.clone()
    bad[0, 0, 0] = float("nan")
    bad[0, 1, 1, 5] = float("inf")
    bad[0, 20, 0, 7] = float("nan")
    lse = torch.empty((1, b.T, 2), device=DEV)
    d = B.btq_kv_attention(bad, starts, lengths, tb, cache, lse=lse).view(1, b.T, 2, 128)
    a = a.view(1, b.T, 2, 128)
    hit = torch.zeros((b.T, 2), dtype=torch.bool)
    hit[0, 0] = hit[1, 1] = hit[20, 0] = True
    assert torch.isnan(d[0, hit]).all() and torch.isnan(lse[0, hit]).all()
    assert torch.equal(d[0, ~hit], a[0, ~hit])


@pytest.mark.gpu
@pytest.mark.parametrize("sigma,q_sigma,scale", [(1.0, 20.0, None), (30.0, 4.0, None), (1e-3, 1.0, None),
                                                 (1.0, 1.0, 1e-6), (1.0, 1.0, 3.0)])
def test_flat_and_sharp_softmax(sigma, q_sigma, scale):
    for n in (6, 7, 8):
        check(BATCHES[n], 1, 4, 1, 128, sigma=sigma, q_sigma=q_sigma, dt=F32, scale=scale)


@pytest.mark.gpu
def test_maximum_that_rises_late():
    # scores grow along the keys, so the sums are rescaled again and again
    D = 64

    def edit(batch, cache):
        for j in range(batch.lengths[0]):
            page, block, t = batch.where(0, j)
            s = np.float32(0.02 * (1 + j) / 4).view(np.uint32) & 0xffff0000
            cache[:, page, :, block, 32 * D + 4 * t:32 * D + 4 * t + 4] = np.frombuffer(
                np.uint32(s | 0x4300).tobytes(), np.uint8)
    check(Batch([1], [900], page=64), 1, 4, 1, D, edit=edit, dt=F32, q_sigma=3.0)
    check(Batch([64], [900], page=64), 1, 2, 1, D, edit=edit, dt=F32, q_sigma=3.0)


@pytest.mark.gpu
@pytest.mark.parametrize("power", [-100, 79])
def test_values_of_any_size(power):
    # scales of values times a power of 2, by every kernel: the same rows times that, to the bit.
    # The first 1024 keys, with which every wave of a block begins, score 7 powers of 2 below
    # the others, which the maximum does not follow: their weights are near 2^7. (Values of
    # 4*2^79 are beyond the 2^80 that is promised.)
    for b, Hq, D in ((Batch([1, 1], [2000, 700], page=64), 4, 64), (Batch([1, 1], [2000, 700], page=64), 4, 160),
                     (Batch([1], [9000], page=64), 5, 64), (Batch([64], [1900], page=64), 8, 64),
                     (Batch([64], [1900], page=64), 8, 160)):
        cache = random_cache(b, 1, 1, D)
        words = cache[..., 32 * D:].view(np.uint32)
        words[..., :32] = 0x3f804300                       # keys: scale 1, z 0
        codes = cache[..., :16 * D]
        codes[:] = 0x11                                    # of ones
        for s in range(b.B):
            for j in range(min(1024, b.lengths[s])):
                page, block, t = b.where(s, j)
                codes[0, page, 0, block, t * D // 2:(t + 1) * D // 2] = 0
        starts, lengths, tb = b.dev()
        q = torch.full((1, b.T, Hq, D), 7 / D / 1.4426950408889634, device=DEV).to(BF16)
        got = []
        for n in (0, power):
            words[..., 32:] += np.uint32((n << 23) & 0xffffffff)
            lse = torch.empty((1, b.T, Hq), device=DEV)
            out = B.btq_kv_attention(q, starts, lengths, tb, torch.from_numpy(cache).to(DEV), scale=1.0,
                                     out_dtype=F32, lse=lse)
            got.append((out, lse))
        assert torch.isfinite(got[1][0]).all() and (got[0][0].abs() > 2.0 ** -9).any()
        assert torch.equal(got[1][0], got[0][0] * 2.0 ** power) and torch.equal(got[1][1], got[0][1])


@pytest.mark.gpu
@pytest.mark.parametrize("shift,gap", [(0, 0), (1, 0), (3, 5), (8, 64), (0, 3)])
def test_query_strides_and_alignment(shift, gap):
    check(BATCHES[7], 2, 4, 2, 64, shift=shift, gap=gap)


@pytest.mark.gpu
def test_same_bits_again_and_in_other_batches():
    out, lse, (q, starts, lengths, tb, cache) = check(BATCHES[7], 2, 4, 1, 128)
    again = B.btq_kv_attention(q, starts, lengths, tb, cache)
    assert torch.equal(again[:, 2:13], out[:, 2:13])
    # the other sequences' contents do not matter
    other = q.clone()
    other[:, 2:5] = 1.0
    part = B.btq_kv_attention(other, starts, lengths, tb, cache)
    assert torch.equal(part[:, 5:13], out[:, 5:13])


@pytest.mark.gpu
def test_long_cache_offsets_pass_32_bits():
    D, page = 128, 64
    per = page // 32 * block_bytes(D)
    pages = (6 << 30) // per
    b = Batch([1], [190], page=page)
    small = torch.from_numpy(random_cache(b, 1, 1, D)).to(DEV)
    q = torch.randn((1, 1, 8, D), device=DEV).to(BF16)
    starts, lengths, tb = b.dev()
    want = B.btq_kv_attention(q, starts, lengths, tb, small)
    cache = torch.zeros((1, pages, 1, page // 32, block_bytes(D)), dtype=torch.uint8, device=DEV)
    far = [pages - 1, (4 << 30) // per, (4 << 30) // per - 1]
    for i, p in enumerate(far):
        cache[0, p] = small[0, int(b.table[0, i])]
    got = B.btq_kv_attention(q, starts, lengths, torch.tensor([far], dtype=torch.int32, device=DEV), cache)
    assert torch.equal(got, want) and want.any()


@pytest.mark.gpu
def test_capture_and_replay():
    # one graph replayed over a growing sequence, whose lengths and pages it reads
    D, page = 128, 64
    b = Batch([1, 1], [2200, 2200], page=page)
    cache = torch.from_numpy(random_cache(b, 2, 1, D)).to(DEV)
    starts, lengths, tb = b.dev()
    q = torch.randn((2, 2, 8, D), device=DEV).to(BF16)
    out = torch.zeros((2, 2, 8 * D), dtype=BF16, device=DEV)
    need = B.btq_kv_attention_workspace_bytes(2, 2, 8, 1, D, 2, tb.shape[1], page)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    assert need > 0
    run = lambda o: B.btq_kv_attention(q, starts, lengths, tb, cache, out=o, workspace=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out)
    for n in (1, 700, 1999, 2000, 0, 513):
        lengths.copy_(torch.tensor([n, max(n - 300, 0)], dtype=torch.int32))
        q.normal_()
        eager = torch.empty_like(out)
        B.btq_kv_attention(q, starts, lengths, tb, cache, out=eager)
        ws.fill_(0xff)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), n


@pytest.mark.gpu
def test_other_stream_and_no_shards():
    b = Batch([1, 3], [800, 50], page=64)
    cache = torch.from_numpy(random_cache(b, 1, 2, 64)).to(DEV)
    q = torch.randn((1, 4, 4, 64), device=DEV).to(BF16)
    starts, lengths, tb = b.dev()
    want = B.btq_kv_attention(q, starts, lengths, tb, cache)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = B.btq_kv_attention(q[0], starts, lengths, tb, cache[0], stream=s)
    s.synchronize()
    assert torch.equal(got, want[0])
    bits = B.btq_kv_attention(q.view(torch.int16), starts, lengths, tb, cache)
    assert bits.dtype == torch.int16 and torch.equal(bits, want.view(torch.int16))
    empty = B.btq_kv_attention(q[:, :0], starts * 0, lengths, tb, cache)
    assert empty.shape == (1, 0, 256)


@pytest.mark.gpu
def test_python_refusals():
    b = Batch([1], [2100], page=64)     # (long enough to need a workspace)
    cache = torch.from_numpy(random_cache(b, 1, 2, 64)).to(DEV)
    q = torch.zeros((1, 1, 4, 64), dtype=BF16, device=DEV)
    starts, lengths, tb = b.dev()
    args = dict(q=q, seq_starts=starts, lengths=lengths, page_table=tb, cache=cache)
    for kw in (dict(q=q[:, :, :3]), dict(q=q[..., :32]), dict(cache=cache[0]), dict(q=q[0]),
               dict(out=torch.zeros((1, 1, 4, 64), dtype=BF16, device=DEV)),
               dict(lse=torch.zeros((1, 1, 2), device=DEV)), dict(seq_starts=starts[1:])):
        with pytest.raises(ValueError):
            B.btq_kv_attention(**{**args, **kw})
    for kw in (dict(q=q.float()), dict(q=q.half()), dict(page_table=tb.long())):
        with pytest.raises(TypeError):
            B.btq_kv_attention(**{**args, **kw})
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(window=-1),
               dict(max_length=-1), dict(workspace=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(RuntimeError):
            B.btq_kv_attention(**{**args, **kw})


# Many columns a sequence, which share the keys that a block stages: the same questions
# once more, with keys in one piece (first two) and in several.
WIDE = [Batch([150], [150]), Batch([70, 1, 0, 200], [300, 90, 5, 200], page=64, before=1, behind=2),
        Batch([50, 1, 90], [200, 900, 90], page=64, slack=1), Batch([33, 280], [1500, 1200], page=128)]


@pytest.mark.gpu
@pytest.mark.parametrize("n", range(len(WIDE)))
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
def test_many_columns(n, D):
    say(f"case: kv attention many columns {n} D={D}")
    check(WIDE[n], 1, 8, 1, D, dt=F32)
    check(WIDE[n], 2, 16, 2, D, causal=n % 2 == 0, window=100, lse=False)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hk", [(5, 1), (17, 1), (40, 2), (12, 4), (64, 1)])
def test_many_columns_in_head_groups(Hq, Hk):
    for n in (1, 2):
        check(WIDE[n], 1, Hq, Hk, 64)


@pytest.mark.gpu
@pytest.mark.parametrize("sigma,q_sigma,scale", [(1.0, 20.0, None), (30.0, 4.0, None), (1.0, 1.0, 3.0)])
def test_many_columns_flat_and_sharp(sigma, q_sigma, scale):
    for n in (1, 3):
        check(WIDE[n], 1, 8, 1, 128, sigma=sigma, q_sigma=q_sigma, dt=F32, scale=scale)


@pytest.mark.gpu
@pytest.mark.parametrize("shift,gap", [(1, 0), (3, 5), (8, 64)])
def test_many_columns_strides_and_alignment(shift, gap):
    check(WIDE[1], 2, 8, 2, 64, shift=shift, gap=gap)


@pytest.mark.gpu
def test_many_columns_missing_pages():
    b = Batch([60, 130], [700, 300], page=32)
    b.table[0, [0, 3, 4, 5, 6, 11]] = -1
    b.table[1, 5] = b.pages
    b.table[1, 2] = -2 ** 31
    check(b, 1, 8, 1, 128)
    check(b, 1, 8, 1, 128, window=60)
    b.table[:] = -1
    out, lse, _ = check(b, 1, 8, 1, 128)
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.gpu
def test_many_columns_nan():
    # a key or value that is NaN reaches the rows that see it, a query that is NaN its row
    D = 64
    b = Batch([160, 50], [180, 60], page=32)
    g = np.random.default_rng(3)
    q = torch.from_numpy(g.standard_normal((1, b.T, 8, D)).astype(np.float32)).to(DEV).to(BF16)
    clean = random_cache(b, 1, 2, D)
    starts, lengths, tb = b.dev()
    a = B.btq_kv_attention(q, starts, lengths, tb, torch.from_numpy(clean).to(DEV))
    assert torch.isfinite(a).all()
    for value in (0, 128):
        dirty = clean.copy()
        page, block, t = b.where(0, 100)
        at = 32 * D + value + 4 * t
        dirty[:, page, :, block, at:at + 4] = np.frombuffer(np.uint32(NAN_WORD).tobytes(), np.uint8)
        d = B.btq_kv_attention(q, starts, lengths, tb, torch.from_numpy(dirty).to(DEV))
        sees = torch.zeros(b.T, dtype=torch.bool)
        sees[80:160] = True                                # row 80 is place 100
        assert torch.isnan(d[0, sees]).all() and torch.equal(d[0, ~sees], a[0, ~sees])
    bad = q.clone()
    bad[0, 20, 3, 7], bad[0, 170, 0, 0] = float("nan"), float("inf")
    d = B.btq_kv_attention(bad, starts, lengths, tb, torch.from_numpy(clean).to(DEV)).view(1, b.T, 8, D)
    hit = torch.zeros((b.T, 8), dtype=torch.bool)
    hit[20, 3] = hit[170, 0] = True
    assert torch.isnan(d[0, hit]).all() and torch.equal(d[0, ~hit], a.view(1, b.T, 8, D)[0, ~hit])


@pytest.mark.gpu
def test_many_columns_captured():
    D, page = 128, 64
    b = Batch([20, 60], [1800, 1800], page=page)
    cache = torch.from_numpy(random_cache(b, 1, 1, D)).to(DEV)
    starts, lengths, tb = b.dev()
    q = torch.randn((1, 80, 8, D), device=DEV).to(BF16)
    out = torch.zeros((1, 80, 8 * D), dtype=BF16, device=DEV)
    need = B.btq_kv_attention_workspace_bytes(1, 80, 8, 1, D, 2, tb.shape[1], page)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    B.btq_kv_attention(q, starts, lengths, tb, cache, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.btq_kv_attention(q, starts, lengths, tb, cache, out=out, workspace=ws)
    for n in (20, 700, 1800, 0, 63):
        lengths.copy_(torch.tensor([n, max(n - 300, 0)], dtype=torch.int32))
        q.normal_()
        eager = torch.empty_like(out)
        B.btq_kv_attention(q, starts, lengths, tb, cache, out=eager)
        ws.fill_(0xff)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager), n


@pytest.mark.gpu
@pytest.mark.parametrize("starts", [[0, 8, 8, 0, 1, 2, 3, 4, 5], [8, 7, 6, 5, 4, 3, 2, 1, 0],
                                    [5, -9, 700, 3, -2 ** 31, 2 ** 31 - 1, 8, 0, 2]])
def test_starts_that_do_not_ascend_stay_inside_the_tensors(starts):
    # the results are unspecified, the guards before and behind them are not (the item
    # search itself is tested in test_item_search.py)
    say(f"case: kv attention starts {starts}")
    # columns of 8 and of 16 in whole groups, equal shares, and many columns in one
    # piece and in several
    for T, Hq, D, length, ml in ((8, 8, 64, 300, 300), (8, 8, 160, 300, 300), (8, 4, 64, 5000, 0),
                                 (130, 8, 64, 300, 300), (300, 8, 128, 5000, 0)):
        b = Batch([T], [length], page=64)
        n = len(starts) - 1
        tb = torch.from_numpy(np.repeat(b.table, n, 0)).to(DEV)
        lengths = torch.full((n,), length, dtype=torch.int32, device=DEV)
        cache = torch.from_numpy(random_cache(b, 1, 1, D)).to(DEV)
        q = torch.randn((1, T, Hq, D), device=DEV).to(BF16)
        st = torch.tensor(starts, dtype=torch.int32, device=DEV)
        room = 1 << 20
        out = torch.full((2 * room + T * Hq * D,), 5.0, device=DEV)
        lse = torch.full((2 * room + T * Hq,), 5.0, device=DEV)
        B.btq_kv_attention(q, st, lengths, tb, cache, max_length=ml,
                           out=out[room:-room].view(1, T, Hq * D), lse=lse[room:-room].view(1, T, Hq))
        torch.cuda.synchronize()
        for x in (out, lse):
            assert (x[:room] == 5).all() and (x[-room:] == 5).all()


@pytest.mark.gpu
@pytest.mark.parametrize("first,last", [(-5, 4), (-2 ** 31, 0), (-40, 2 ** 30)])
def test_starts_outside_the_batch_are_cut(first, last):
    # the same rows as with starts cut to [0,T], by each kernel (as in the test above)
    for new, Hq, D, length, ml in (([3, 2, 3], 1, 64, 300, 300), ([3, 2, 3], 16, 160, 300, 300),
                                   ([3, 2, 3], 4, 64, 5000, 0), ([30, 90, 10], 8, 64, 300, 300),
                                   ([100, 30, 170], 8, 128, 5000, 0)):
        b = Batch(new, [length, length - 7, 200], page=64)
        starts, lengths, tb = b.dev()
        cache = torch.from_numpy(random_cache(b, 1, 1, D)).to(DEV)
        q = torch.randn((1, b.T, Hq, D), device=DEV).to(BF16)
        wide = starts.clone()
        wide[0] = first
        wide[-1] += last
        got = []
        for st in (starts, wide):
            out = torch.full((1, b.T, Hq * D), 5.0, device=DEV)
            lse = torch.full((1, b.T, Hq), 5.0, device=DEV)
            B.btq_kv_attention(q, st, lengths, tb, cache, max_length=ml, out=out, lse=lse)
            got.append((out, lse))
        assert not (got[0][0] == 5).any()
        assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


# ---- CPU: all return before any HIP call ---------------------------------------

A = 0x10000
OK, ARG, SHAPE, ALIGN = _lib.BTQ_OK, _lib.BTQ_ERR_ARG, _lib.BTQ_ERR_SHAPE, _lib.BTQ_ERR_ALIGN


def call(q=A, qs=0, qp=1024, qh=128, P=1, T=4, Hq=8, Hk=2, D=128, starts=A, lengths=A, nb=1, tb=A,
         mp=2, cache=A, pages=4, size=64, scale=0.1, causal=1, window=0, ml=0, out=A, ot=1, lse=A,
         ws=A, wsb=1 << 40):
    return _lib.load().btq_kv_attention(q, qs, qp, qh, P, T, Hq, Hk, D, starts, lengths, nb, tb, mp,
                                        cache, pages, size, scale, causal, window, ml, out, ot, lse,
                                        ws, wsb, None)


def test_refusals():
    assert call(T=0) == OK and call(nb=0) == OK
    for kw in (dict(P=0), dict(P=65536), dict(T=-1), dict(Hk=0), dict(Hq=0), dict(Hq=7), dict(Hq=65536),
               dict(D=48), dict(D=320), dict(nb=-1), dict(mp=-1), dict(mp=1 << 25), dict(size=33),
               dict(size=1 << 17), dict(pages=0), dict(pages=1 << 31), dict(qp=-1), dict(qh=-1),
               dict(P=2, qs=-1), dict(qp=1 << 61), dict(window=-1), dict(ml=-1), dict(ml=1 << 31),
               dict(T=1 << 28, Hq=16)):
        assert call(**kw) == SHAPE, kw
    for kw in (dict(q=None), dict(out=None), dict(starts=None), dict(lengths=None), dict(tb=None),
               dict(cache=None), dict(ot=2), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("inf")), dict(scale=1.8e38), dict(scale=float("nan"))):
        assert call(**kw) == ARG, kw
    for kw in (dict(q=A + 1), dict(out=A + 2), dict(ot=0, out=A + 4), dict(lse=A + 2), dict(ws=A + 8),
               dict(cache=A + 8), dict(starts=A + 1)):
        assert call(**kw) == ALIGN, kw
    assert call(mp=1 << 12, ws=None) == ARG
    assert call(mp=1 << 12, wsb=0) == _lib.BTQ_ERR_WORKSPACE


def test_workspace_bytes():
    f = _lib.load().btq_kv_attention_workspace_bytes
    assert f(1, 1, 8, 1, 128, 1, 2, 64, 0) == 0                 # short: one split
    n = f(1, 1, 8, 1, 128, 1, 1 << 12, 64, 0)
    assert n > 0 and f(1, 1, 8, 1, 128, 1, 1 << 12, 64, 1 << 29) == n
    assert f(1, 1, 8, 1, 128, 1, 1 << 12, 64, 100) == 0         # the bound says short
    for bad in ((0, 1, 8, 1, 128, 1, 2, 64, 0), (1, 1, 8, 3, 128, 1, 2, 64, 0),
                (1, 1, 8, 1, 100, 1, 2, 64, 0), (1, 1, 8, 1, 128, 1, 2, 40, 0),
                (1, 1, 8, 1, 128, 1, 2, 64, -1), (1, 0, 8, 1, 128, 1, 2, 64, 0)):
        assert f(*bad) == 0
