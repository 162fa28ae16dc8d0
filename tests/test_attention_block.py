"""The attention group run together, as a transformer block uses it: in a decode loop
over one cache, in captured graphs, on two streams at once, and by tp_block.py."""
import json
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import bit_tensor_activation_amd as B
import tp_block
from helpers import say
from kv_helpers import BF16, DEV, F32, Batch, attention, block_bytes, host, random_cache, table

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Decoder:
    """Projected rows of a few sequences, taken through head norm, append and attention."""

    def __init__(self, P=2, nseq=3, Hq=4, Hk=1, D=64, page=32, longest=150, seed=0):
        self.P, self.n, self.Hq, self.Hk, self.D, self.page = P, nseq, Hq, Hk, D, page
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.rows = torch.randn((P, nseq, longest, Hq + 2 * Hk, D), generator=g, device=DEV).to(BF16)
        pages = -(-longest // page)
        self.table = torch.randperm(nseq * pages, generator=g, device=DEV).int().view(nseq, pages)
        self.cache = torch.zeros((P, nseq * pages, Hk, page // 32, block_bytes(D)),
                                 dtype=torch.uint8, device=DEV)
        self.cos, self.sin = table(longest, D)
        self.qw = 1 + 0.1 * torch.randn(D, generator=g, device=DEV)
        self.kw = 1 + 0.1 * torch.randn(D, generator=g, device=DEV)

    def step(self, qkv, starts, lengths, positions, stream=None, **kw):
        H = self.Hq + self.Hk
        qk = B.btq_head_norm_rope(qkv[:, :, :H], self.Hq, q_weight=self.qw, k_weight=self.kw,
                                  positions=positions, cos=self.cos, sin=self.sin, stream=stream)
        B.btq_kv_append(qk[:, :, self.Hq:], qkv[:, :, H:].contiguous(), starts, lengths, self.table,
                        self.cache, stream=stream)
        return B.btq_kv_attention(qk[:, :, :self.Hq], starts, lengths, self.table, self.cache,
                                  stream=stream, **kw)

    def batch(self, done, new):
        """The next new[b] rows of every sequence of which done[b] are cached."""
        rows = torch.cat([self.rows[:, b, done[b]:done[b] + new[b]] for b in range(self.n)], 1)
        pos = np.concatenate([np.arange(d, d + n) for d, n in zip(done, new)])
        return (rows, torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV),
                torch.tensor([d + n for d, n in zip(done, new)], dtype=torch.int32, device=DEV),
                torch.tensor(pos, dtype=torch.int32, device=DEV))


@pytest.mark.gpu
def test_decode_loop_gives_the_rows_of_one_prefill():
    # token by token, and by drafts of 3, against all at once: the same cache bytes
    # and, to the order of sums and the rounding of weights, the same rows
    longest = 150
    one, many = Decoder(longest=longest), Decoder(longest=longest)
    whole = one.step(*one.batch([0] * 3, [longest] * 3), out_dtype=F32)
    done, rows = [0, 0, 0], []
    while done[0] < longest:
        new = [min(n, longest - d) for n, d in zip(((100, 20, 1) if done[0] == 0 else (1, 3, 2)), done)]
        if sum(new) == 0:
            break
        got = many.step(*many.batch(done, new), out_dtype=F32)
        at = 0
        for b, n in enumerate(new):
            for i in range(n):
                rows.append((b * longest + done[b] + i, got[:, at + i]))
            at += n
        done = [d + n for d, n in zip(done, new)]
    for b in range(3):      # what is left of the others
        if done[b] < longest:
            new = [0, 0, 0]
            new[b] = longest - done[b]
            got = many.step(*many.batch(done, new), out_dtype=F32)
            rows += [(b * longest + done[b] + i, got[:, i]) for i in range(new[b])]
            done[b] = longest
    assert torch.equal(one.cache, many.cache)
    assert sorted(r for r, _ in rows) == list(range(3 * longest))
    # |v| is below 6 here; weights are rounded to bf16 on both sides
    assert all((got - whole[:, r]).abs().max() <= 2 * 2.0 ** -8 * 6 for r, got in rows)


@pytest.mark.gpu
def test_captured_decode_step_over_a_growing_sequence():
    d = Decoder(longest=140)
    e = Decoder(longest=140)
    start = [100, 3, 64]
    for x in (d, e):
        x.step(*x.batch([0, 0, 0], start))
    qkv, starts, lengths, pos = d.batch(start, [1, 1, 1])
    qkv, out = qkv.contiguous(), torch.empty((2, 3, 4 * 64), dtype=BF16, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        d.step(qkv, starts, lengths, pos, out=out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.step(qkv, starts, lengths, pos, out=out)
    for i in range(6):
        now = [n + i for n in start]
        rows, _, ln, ps = e.batch(now, [1, 1, 1])
        want = e.step(rows, starts, ln, ps)
        qkv.copy_(rows)
        lengths.copy_(ln)
        pos.copy_(ps)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i
        assert torch.equal(d.cache, e.cache)


@pytest.mark.gpu
def test_two_streams_at_once():
    # calls on two streams with their own caches, outputs and workspaces do not meet
    a, b = Decoder(seed=1, longest=2300), Decoder(seed=2, longest=2300)
    plain = [Decoder(seed=1, longest=2300), Decoder(seed=2, longest=2300)]
    new = [2200, 40, 7]
    want = [x.step(*x.batch([0, 0, 0], new)) for x in plain]
    again = [x.step(*x.batch(new, [1, 1, 1])) for x in plain]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    batches = [(x.batch([0, 0, 0], new), x.batch(new, [1, 1, 1])) for x in (a, b)]
    torch.cuda.synchronize()
    got = [[], []]
    for step in range(2):
        for i, x in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append(x.step(*batches[i][step]))
    torch.cuda.synchronize()
    for i, x in enumerate((a, b)):
        assert torch.equal(got[i][0], want[i]) and torch.equal(got[i][1], again[i])
        assert torch.equal(x.cache, plain[i].cache)


@pytest.mark.gpu
def test_stream_argument_orders_the_calls_it_makes():
    a, b = Decoder(seed=3), Decoder(seed=3)
    want = a.step(*a.batch([0, 0, 0], [100, 1, 30]))
    batch = b.batch([0, 0, 0], [100, 1, 30])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = b.step(*batch, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    raw = b.step(*batch, stream=int(s.cuda_stream))
    s.synchronize()
    assert torch.equal(raw, want)


@pytest.mark.gpu
def test_sequences_that_share_pages():
    # a prefix held once: two sequences name its pages, each has its own last one
    D, b = 64, Batch([1, 1], [140, 150], page=64)
    b.table[1, :2] = b.table[0, :2]
    cache = random_cache(b, 1, 1, D)
    q = torch.randn((1, 2, 4, D), device=DEV).to(BF16)
    starts, lengths, tb = b.dev()
    out = B.btq_kv_attention(q, starts, lengths, tb, torch.from_numpy(cache).to(DEV), out_dtype=F32)
    want, tol, _, _ = attention(b, cache, host(q), 1, D, D ** -0.5)
    assert (np.abs(host(out).reshape(want.shape) - want) <= 1.05 * tol + 2.0 ** -24 * np.abs(want)).all()


@pytest.mark.gpu
def test_splits_of_one_context_merge_by_their_sums():
    # two halves of a sequence attended to apart, joined by lse: the whole, to the
    # rounding of both parts' weights (2^-8 of the values, which are below 6)
    D, L = 128, 3000
    b = Batch([1], [L], page=64)
    cache = torch.from_numpy(random_cache(b, 1, 1, D)).to(DEV)
    q = torch.randn((1, 1, 8, D), device=DEV).to(BF16)
    starts, lengths, tb = b.dev()
    parts = []
    for first, n in ((0, 1408), (1408, L - 1408)):
        lse = torch.empty((1, 1, 8), device=DEV)
        t = tb[:, first // 64:].contiguous()
        o = B.btq_kv_attention(q, starts, torch.full_like(lengths, n), t, cache, causal=False,
                               out_dtype=F32, lse=lse)
        parts.append((o.view(8, D).double(), lse.view(8, 1).double()))
    total = torch.logaddexp(parts[0][1], parts[1][1])
    joined = sum(o * torch.exp(l - total) for o, l in parts)
    whole = B.btq_kv_attention(q, starts, lengths, tb, cache, causal=False, out_dtype=F32)
    assert (joined - whole.view(8, D)).abs().max() <= 2 * 2.0 ** -8 * 6


@pytest.mark.gpu
def test_no_memory_for_what_a_call_makes():
    # refused by torch's allocator, at a hundredth of the card, as a call of torch's is
    d = Decoder()
    qkv, starts, lengths, pos = d.batch([0, 0, 0], [2, 1, 1])
    d.step(qkv, starts, lengths, pos)
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(0.01)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            B.btq_kv_gather(starts, lengths, d.table, d.cache, tokens=1 << 25)
        big = qkv[:, :1, :d.Hq].expand(2, 1 << 24, d.Hq, d.D)
        with pytest.raises(torch.OutOfMemoryError):
            B.btq_head_norm_rope(big, d.Hq)
        with pytest.raises(torch.OutOfMemoryError):
            B.btq_kv_attention(big, starts, lengths, d.table, d.cache)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    d.step(qkv, starts, lengths, pos)


@pytest.mark.gpu
def test_tp_block_with_attention():
    s = tp_block.prepare(2, 12, 256, 256, 192, 8)
    tp_block.prepare_attention(s, 3, 70, 1)
    x = tp_block.attend(s)
    assert x.shape == (2, 12, 256) and torch.isfinite(x.view(BF16)).all()
    again = tp_block.attend(s)          # the same places are written again
    assert torch.equal(x, again)
    # 8-bit codes of the projection: q is off by under 2%, scores by under 0.1
    err = tp_block.relative_error(x.view(BF16), tp_block.exact_attention(s))
    say(f"  error of x {err}")
    assert err < 0.1
    s["x"] = x.view(BF16)
    y, residual, z = tp_block.step(s)
    assert torch.isfinite(y).all() and torch.isfinite(residual.float()).all() and torch.isfinite(z.float()).all()


@pytest.mark.gpu
@pytest.mark.parametrize("cached", [70, 0])
def test_tp_block_error_of_attention(cached):
    s = tp_block.prepare(2, 12, 256, 256, 192, 8)
    tp_block.prepare_attention(s, 3, cached, 1)
    x = tp_block.attend(s).view(BF16)
    # Over the cache as it is: activations and weights in 8 bits, of rows of 256 normal values
    # up to 4.2, are off by 4.2/127/sqrt(12) = 0.0095 each, queries by 0.0135, and so scores
    # (keys have 1 in the mean square) and rows; three roundings to bf16 add 0.003.
    err = tp_block.relative_error(x, tp_block.exact_attention(s))
    # Over the rows before their codes, projection, norm, rotation and places among what is
    # compared: steps of up to 7/15 for 128 normal values, off by 7/15/sqrt(12) = 0.135, by keys
    # and by values.
    rows = tp_block.relative_error(x, tp_block.exact_attention(s, cached=False))
    say(f"  error of x {err}, against rows {rows}")
    assert err <= 0.02 and rows <= 0.2


@pytest.mark.gpu
def test_tp_block_command_with_attention():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "tp_block.py"), "--P", "2", "--T", "6", "--H",
                        "256", "--K", "256", "--N", "128", "--k", "8", "--steps", "2", "--cached", "40",
                        "--B", "2"], capture_output=True, text=True, timeout=100, cwd=ROOT)
    assert r.returncode == 0, r.stderr
    out = json.loads(r.stdout.strip().splitlines()[-1])
    assert out["config"]["cached"] == 40 and out["attention_us"] > 0 and out["relative_error"]["x"] < 0.1


def test_attention_needs_sizes_that_fit():
    s = dict(P=1, T=4, H=64, K=100)
    with pytest.raises(ValueError):
        tp_block.prepare_attention(s, 2, 10, 1)
