"""One tensor-parallel boundary of a transformer, end to end on the GPU.

From the activations of a row-parallel layer to the next block's first
product, with every step in the library's HIP kernels:

    x [P,T,K] --btq_int8_linear--> partial sums [P,T,H]      (P shards)
      --btq_compress_pack--> int4/BF16 messages               (sender)
      --btq_decompress_reduce--> y [T,H]                      (receiver)
      --btq_block_norm--> residual [T,H], 8-bit rows [T,H]    (norms, gate)
      --btq_int8_matmul--> z [P,T,N]                          (next block)

Weights and activations are random; the weights get their 8-bit codes and the
codec its calibration once, before the step. The script times the step and
each call of it, and measures y, the residual and z against the same layer
computed from the unquantized values in float64.

With --cached C the activations x come from the attention before that layer: B
sequences, each with C tokens in a paged 4-bit cache, of which T/B new ones go
through the block. Every shard has K/D query heads and --kv_heads key heads:

    h [T,H] --btq_int8_linear--> queries, keys, values [P,T,heads,D]
      --btq_head_norm_rope--> norm and rotation, in place
      --btq_kv_append--> cache       --btq_kv_attention--> x [P,T,K]

and the script measures x against attention in float64 over what the cache holds, and over
the keys and values before they were quantized.

    python tp_block.py                        # P=8 T=2048 H=4096 K=512 N=2048
    python tp_block.py --T 8 --H 8192 --K 1024 --N 1024
    python tp_block.py --T 32 --H 8192 --K 1024 --N 1024 --cached 2000 --B 32

It prints one JSON line.
"""
from __future__ import annotations

import argparse
import json
import sys

import torch

import bit_tensor_activation_amd as B

EPS = 1e-6


def prepare(P: int, T: int, H: int, K: int, N: int, k: int, seed: int = 1,
            calib_batches: int = 4) -> dict:
    """Weights, calibrated codec and one batch of inputs."""
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def rnd(*shape):
        return torch.randn(shape, generator=g, device=dev)
    s = dict(P=P, T=T, H=H, K=K, N=N, k=k)
    s["w1_exact"] = rnd(P, H, K) * (P * K) ** -0.5     # y of unit variance
    # a few output features are wide on every shard: the codec's outliers
    wide = torch.randperm(H, generator=g, device=dev)[:k // 2]
    s["w1_exact"][:, wide] *= 30.0
    s["w2_exact"] = rnd(P, N, H) * H ** -0.5
    s["w1"], s["w1_scale"] = B.btq_quantize_rows(s["w1_exact"])
    s["w2"], s["w2_scale"] = B.btq_quantize_rows(s["w2_exact"])
    s["post_weight"], s["pre_weight"] = 1 + 0.1 * rnd(H), 1 + 0.1 * rnd(H)
    s["gate"] = torch.tanh(rnd(1, H))

    run_min = torch.empty((P, H), dtype=torch.float32, device=dev)
    run_max = torch.empty_like(run_min)
    for b in range(calib_batches):
        x = rnd(P, max(T, 256), K).to(torch.bfloat16)
        B.btq_calib_update(B.btq_int8_linear(x, s["w1"], s["w1_scale"]), run_min, run_max, 0.9,
                           b == 0)
    s["sel"] = B.btq_select_outliers(run_min, run_max, k)
    s["x"] = rnd(P, T, K).to(torch.bfloat16)
    s["residual"] = rnd(T, H).to(torch.bfloat16)
    return s


def prepare_attention(s: dict, B_: int, cached: int, kv_heads: int, D: int = 128,
                      page: int = 64, seed: int = 2) -> None:
    """Adds to s what the attention before the block needs: B_ sequences whose pages
    hold `cached` random tokens each, and the projection of their new ones."""
    P, T, H, K = s["P"], s["T"], s["H"], s["K"]
    if K % D or T % B_:
        raise ValueError("K must be a multiple of D, and T of the sequences")
    dev = s["residual"].device
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def rnd(*shape):
        return torch.randn(shape, generator=g, device=dev)
    n, heads = T // B_, K // D
    s["heads"], s["kv_heads"], s["D"], s["length"] = heads, kv_heads, D, cached + n
    s["w0_exact"] = rnd(P, (heads + 2 * kv_heads) * D, H) * H ** -0.5
    s["w0"], s["w0_scale"] = B.btq_quantize_rows(s["w0_exact"])
    s["h"] = rnd(T, H).to(torch.bfloat16)
    s["q_weight"], s["k_weight"] = 1 + 0.1 * rnd(D), 1 + 0.1 * rnd(D)
    freq = 10000.0 ** (-torch.arange(0, D, 2, device=dev, dtype=torch.float64) / D)
    angle = torch.arange(s["length"], device=dev, dtype=torch.float64)[:, None] * freq
    s["cos"], s["sin"] = torch.cos(angle).float(), torch.sin(angle).float()

    pages = -(-s["length"] // page)
    s["table"] = torch.randperm(B_ * pages, generator=g, device=dev).int().view(B_, pages)
    s["cache"] = torch.zeros((P, B_ * pages, kv_heads, page // 32, B.btq_kv_block_bytes(D)),
                             dtype=torch.uint8, device=dev)
    s["starts"] = torch.arange(0, T + 1, n, device=dev, dtype=torch.int32)
    s["lengths"] = torch.full((B_,), s["length"], dtype=torch.int32, device=dev)
    s["positions"] = (torch.arange(T, device=dev) % n + cached).int()
    if cached:
        old = torch.arange(0, B_ * cached + 1, cached, device=dev, dtype=torch.int32)
        s["kv"] = kv = rnd(2, P, B_ * cached, kv_heads, D).to(torch.bfloat16)
        B.btq_kv_append(kv[0], kv[1], old, torch.full_like(s["lengths"], cached), s["table"],
                        s["cache"])


def attend(s):
    """x [P,T,K] of the new tokens, which are in the cache after it."""
    P, T, D, Hq, Hk = s["P"], s["T"], s["D"], s["heads"], s["kv_heads"]
    qkv = B.btq_int8_linear(s["h"], s["w0"], s["w0_scale"]).view(P, T, Hq + 2 * Hk, D)
    qk = qkv[:, :, :Hq + Hk]
    B.btq_head_norm_rope(qk, Hq, q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                         positions=s["positions"], cos=s["cos"], sin=s["sin"], out=qk)
    B.btq_kv_append(qk[:, :, Hq:], qkv[:, :, Hq + Hk:], s["starts"], s["lengths"], s["table"],
                    s["cache"])
    return B.btq_kv_attention(qk[:, :, :Hq], s["starts"], s["lengths"], s["table"], s["cache"],
                              max_length=s["length"])


def exact_attention(s, cached: bool = True):
    """x in float64 from the unquantized projection. The keys and values are those that
    the cache holds, or, without `cached`, the rows that were put there before they were
    quantized, those of the new tokens from the projection."""
    P, T, D, Hq, Hk = s["P"], s["T"], s["D"], s["heads"], s["kv_heads"]
    seqs, L = len(s["lengths"]), s["length"]
    n = T // seqs
    c, sn = (s[t][s["positions"].long()].double()[:, None] for t in ("cos", "sin"))

    def project(p, first, heads, weight=None):
        y = s["h"].double() @ s["w0_exact"][p, first * D:(first + heads) * D].double().t().contiguous()
        y = y.view(T, heads, D)
        if weight is None:
            return y
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * weight.double()
        a, b = y[..., :D // 2], y[..., D // 2:]
        return torch.cat((a * c - b * sn, b * c + a * sn), -1)

    def rows(p):
        """Keys and values [seqs,L,Hk,D]."""
        new = (project(p, Hq, Hk, s["k_weight"]), project(p, Hq + Hk, Hk))
        new = [x.view(seqs, n, Hk, D) for x in new]
        if L == n:
            return new
        return [torch.cat((o[p].double().view(seqs, L - n, Hk, D), x), 1) for o, x in zip(s["kv"], new)]
    if cached:
        every = torch.arange(0, seqs * L + 1, L, device=s["h"].device, dtype=torch.int32)
        k, v = (x.view(P, seqs, L, Hk, D) for x in B.btq_kv_gather(
            every, s["lengths"], s["table"], s["cache"], tokens=seqs * L, dtype=torch.float32))
    seen = (torch.arange(L, device=s["h"].device) <= torch.arange(L - n, L, device=s["h"].device)[:, None])
    out = []
    for p in range(P):
        q = project(p, 0, Hq, s["q_weight"])
        kp, vp = (k[p].double(), v[p].double()) if cached else rows(p)
        x = []
        for i in range(seqs):
            for h in range(Hq):
                kk, vv = (u[i, :, h // (Hq // Hk)] for u in (kp, vp))
                t = q[i * n:(i + 1) * n, h] @ kk.t().contiguous() * D ** -0.5
                x.append(torch.softmax(t.masked_fill(~seen, -float("inf")), -1) @ vv)
        out.append(torch.stack(x).view(seqs, Hq, n, D).transpose(1, 2).reshape(T, Hq * D))
    return torch.stack(out)


def linear(s):
    return B.btq_int8_linear(s["x"], s["w1"], s["w1_scale"])


def send(s, sums):
    c = s["sel"]
    return B.btq_compress_pack(sums, s["k"], c["rscale"], c["zero_point"], c["outlier_idx"],
                               c["cmap"])


def receive(s, packed, outliers):
    c = s["sel"]
    return B.btq_decompress_reduce(packed, outliers, s["H"], c["scale"], c["zero_point"], c["fmap"])


def norm(s, y):
    return B.btq_block_norm(y, s["residual"], post="rms", post_weight=s["post_weight"],
                            gate=s["gate"], pre="rms", pre_weight=s["pre_weight"], eps=EPS,
                            n_dtype=torch.int8)


def project(s, q, q_scale):
    return B.btq_int8_matmul(q, q_scale, s["w2"], s["w2_scale"])


def step(s):
    """(y, residual, z) of one batch."""
    y = receive(s, *send(s, linear(s)))
    residual, q, q_scale = norm(s, y)
    return y, residual, project(s, q, q_scale).view(torch.bfloat16)


def exact(s):
    """The same (y, residual, z) from the unquantized values, in float64."""
    def rms(v, w):
        return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * w.double()
    y = sum(s["x"][p].double() @ s["w1_exact"][p].double().t().contiguous()
            for p in range(s["P"]))
    r = s["residual"].double() + s["gate"].double() * rms(y, s["post_weight"])
    n = rms(r, s["pre_weight"])
    z = torch.stack([n @ s["w2_exact"][p].double().t().contiguous() for p in range(s["P"])])
    return y, r, z


def relative_error(got, want) -> float:
    return float((got.double() - want).norm() / want.norm())


def time_us(fn, steps: int) -> float:
    for _ in range(3):
        fn()
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(steps):
        fn()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / steps * 1e3


def main() -> int:
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("P", 8), ("T", 2048), ("H", 4096), ("K", 512), ("N", 2048), ("k", 64),
                        ("steps", 50), ("cached", -1), ("B", 1), ("kv_heads", 1)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    if not torch.cuda.is_available():
        print("tp_block.py needs a GPU (every step runs in HIP kernels)", file=sys.stderr)
        return 2
    s = prepare(a.P, a.T, a.H, a.K, a.N, a.k)
    got, want = step(s), exact(s)
    sums = linear(s)
    message = send(s, sums)
    y = receive(s, *message)
    _, q, q_scale = norm(s, y)
    calls = {"int8_linear": lambda: linear(s), "compress_pack": lambda: send(s, sums),
             "decompress_reduce": lambda: receive(s, *message), "block_norm": lambda: norm(s, y),
             "int8_matmul": lambda: project(s, q, q_scale)}
    if a.cached >= 0:
        prepare_attention(s, a.B, a.cached, a.kv_heads)
        s["x"] = attend(s).view(torch.bfloat16)
        print(json.dumps({
            "config": {**{n: s[n] for n in "PTHKNk"}, "B": a.B, "cached": a.cached,
                       "heads": s["heads"], "kv_heads": s["kv_heads"]},
            "attention_us": round(time_us(lambda: attend(s), a.steps), 1),
            "step_us": round(time_us(lambda: (s.update(x=attend(s)), step(s)), a.steps), 1),
            # against attention over the cache as it is, and over the rows before their codes
            "relative_error": {name: round(relative_error(s["x"].view(torch.bfloat16), exact_attention(s, cached)), 5)
                               for name, cached in (("x", True), ("x_rows", False))}}))
        return 0
    print(json.dumps({
        "config": {n: s[n] for n in "PTHKNk"},
        "step_us": round(time_us(lambda: step(s), a.steps), 1),
        "calls_us": {n: round(time_us(f, a.steps), 1) for n, f in calls.items()},
        "relative_error": {n: round(relative_error(g, w), 5)
                           for n, g, w in zip(("y", "residual", "z"), got, want)}}))
    return 0


if __name__ == "__main__":
    sys.exit(main())
