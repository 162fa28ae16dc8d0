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

    python tp_block.py                        # P=8 T=2048 H=4096 K=512 N=2048
    python tp_block.py --T 8 --H 8192 --K 1024 --N 1024

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
                        ("steps", 50)):
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
    print(json.dumps({
        "config": {n: s[n] for n in "PTHKNk"},
        "step_us": round(time_us(lambda: step(s), a.steps), 1),
        "calls_us": {n: round(time_us(f, a.steps), 1) for n, f in calls.items()},
        "relative_error": {n: round(relative_error(g, w), 5)
                           for n, g, w in zip(("y", "residual", "z"), got, want)}}))
    return 0


if __name__ == "__main__":
    sys.exit(main())
