"""The measured cases of the operators around the codec: the block norm that
reads the receiver's output, and the 8-bit linear layer that makes the
sender's partial sums.

Three paths, chosen by a case's "op":
  norm    btq_block_norm: u = post(y), r' = r + alpha*gate*u, n = pre(r').
  linear  btq_int8_linear: each token row of x gets 8-bit codes and a scale,
          then y[p,t,n] = sum_k codes[p,t,k]*w[p,n,k] * a_scale * w_scale.
  step    btq_block_norm with 8-bit output, then btq_int8_matmul of those
          rows by every shard's weights (a column-parallel layer).

Sizes are those of the codec's own workloads (P shards, T tokens, H features)
with K = H/P for an attention output and K = 4H/P for the second product of a
feed-forward layer; the ragged ones are generic.
"""
from __future__ import annotations

import torch

own = False

NORM_EPS = 1e-6
MAX_FLOPS = 2 * 4 * 8192 * 8192 * 8192     # the largest listed product
MAX_NORM = 16384 * 8192                    # the largest listed norm, elements
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _norm(name, T, H, y, residual, post="rms", pre="rms", gate="none", gate_rows=0, alpha=1.0,
          n="bf16"):
    case = dict(op="norm", T=T, H=H, y=y, residual=residual, post=post, pre=pre, gate=gate,
                gate_rows=gate_rows, alpha=alpha, n=n)
    return dict(case, name=name) if name else case


def _linear(name, P, T, K, N, y="bf16", bias=False):
    case = dict(op="linear", P=P, T=T, K=K, N=N, y=y, bias=bias)
    return dict(case, name=name) if name else case


def _step(name, P, T, H, N, y="f32", residual="bf16"):
    case = dict(op="step", P=P, T=T, H=H, N=N, y=y, residual=residual)
    return dict(case, name=name) if name else case


def listed():
    return [
        # one token of a decode: latency
        _norm("norm decode 1", 1, 8192, "f32", "bf16"),
        # a decode batch behind the bf16-output receiver, with a learned gate per feature
        _norm("norm decode 64", 64, 8192, "bf16", "bf16", gate="f32", gate_rows=1, alpha=0.5),
        # odd sizes, layer norms, a gate for every token and feature, fp32 residual
        _norm("norm ragged layer", 333, 1001, "f32", "f32", post="layer", pre="layer",
              gate="bf16", gate_rows=333, n="f32"),
        # prefill of 8 sequences, each with its own gate
        _norm("norm prefill 2048", 2048, 4096, "f32", "bf16", gate="bf16", gate_rows=8),
        # the longest batch of the codec's workloads
        _norm("norm stress 16384", 16384, 8192, "f32", "bf16", alpha=0.25),
        # attention output of one decoded token, all 8 shards: weights once through, latency
        _linear("linear decode 1", 8, 1, 1024, 8192),
        # second feed-forward product of a decode batch: weights from HBM
        _linear("linear decode 64", 8, 64, 4096, 8192),
        # odd sizes in every direction, fp32 output, bias
        _linear("linear ragged", 3, 77, 1000, 999, y="f32", bias=True),
        # attention output of a prefill: short sums, many outputs
        _linear("linear prefill 2048", 8, 2048, 512, 4096),
        # second feed-forward product of a long prefill: matrix rate
        _linear("linear prefill 8192", 4, 8192, 8192, 8192),
        # decode: norm to 8 bits, then every shard's slice of the next projection
        _step("step decode 8", 8, 8, 8192, 1024),
        # the same for a prefill into the first feed-forward product
        _step("step prefill 2048", 8, 2048, 4096, 2048, y="bf16"),
    ]


def _size(rng, lo, hi, multiple):
    """Log-uniform in [lo, hi]; two thirds of the draws are rounded to `multiple`."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    if rng.random() < 2 / 3 and v > multiple:
        v = v // multiple * multiple
    return v + 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(("norm", "linear", "step"))
    T = _size(rng, 1, 16384, 8)
    if op == "norm":
        H = _size(rng, 256, 8192, 64)
        kind = rng.choice(("rms", "rms", "layer"))
        gate = rng.choice(("none", "f32", "bf16"))
        rows = 0 if gate == "none" else rng.choice((1, T))
        return _norm(None, T, H, rng.choice(("f32", "bf16")), rng.choice(("bf16", "bf16", "f32")),
                     post=rng.choice((kind, kind, "none")), pre=kind, gate=gate, gate_rows=rows,
                     alpha=rng.choice((1.0, 0.5, 0.125)), n=rng.choice(("bf16", "bf16", "f32")))
    P = rng.choice((1, 2, 3, 4, 8))
    if op == "linear":
        K = _size(rng, 64, 8192, 64)
        N = _size(rng, 256, 8192, 64)
        T = max(1, min(T, MAX_FLOPS // (2 * P * K * N), (1 << 29) // (P * N)))
        return _linear(None, P, T, K, N, y=rng.choice(("bf16", "bf16", "f32")),
                       bias=rng.random() < 0.25)
    H = _size(rng, 256, 8192, 64)
    N = _size(rng, 256, 4096, 64)
    T = max(1, min(T, MAX_FLOPS // (2 * P * H * N), (1 << 29) // (P * N)))
    return _step(None, P, T, H, N, y=rng.choice(("f32", "bf16")))


# ---- inputs -----------------------------------------------------------------

def _normal(g, shape, dev, sigma=1.0):
    return torch.randn(shape, generator=g, device=dev) * sigma


def _widen(v, g, dev, factor):
    """A few features have wide ranges, the same ones for every token."""
    H = v.shape[-1]
    cols = torch.randint(0, H, (max(1, H // 200),), generator=g, device=dev)
    v[..., cols] *= factor
    return v


def _weights(g, P, N, K, dev):
    """8-bit weights [P,N,K] and the scale of each channel [P,N]."""
    w = torch.empty((P, N, K), dtype=torch.int8, device=dev)
    for p in range(P):
        w[p] = _normal(g, (N, K), dev, 32.0).round_().clamp_(-127, 127).to(torch.int8)
    s = (0.5 + torch.rand((P, N), generator=g, device=dev)) * (0.02 / 32.0)
    return w, s


def _norm_inputs(case, g, dev):
    T, H = case["T"], case["H"]
    s = {"y": _widen(_normal(g, (T, H), dev, 0.5), g, dev, 30.0).to(DTYPES[case["y"]]),
         "residual": _widen(_normal(g, (T, H), dev, 2.0), g, dev, 10.0).to(DTYPES[case["residual"]]),
         "post_weight": 1.0 + _normal(g, (H,), dev, 0.1), "pre_weight": 1.0 + _normal(g, (H,), dev, 0.1),
         "post_bias": None, "pre_bias": None, "gate": None}
    if case.get("post", "rms") == "layer":
        s["post_bias"] = _normal(g, (H,), dev, 0.1)
    if case.get("pre", "rms") == "layer":
        s["pre_bias"] = _normal(g, (H,), dev, 0.1)
    if case.get("post", "rms") == "none":
        s["post_weight"] = None
    if case.get("gate", "none") != "none":
        s["gate"] = torch.tanh(_normal(g, (case["gate_rows"], H), dev)).to(DTYPES[case["gate"]])
    s["residual_out"] = torch.empty_like(s["residual"])
    return s


def prepare(case, seed):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    s = {"case": case}
    if case["op"] in ("norm", "step"):
        s.update(_norm_inputs(case, g, dev))
    if case["op"] == "norm":
        s["n"] = torch.empty(s["y"].shape, dtype=DTYPES[case["n"]], device=dev)
        return s
    P, T, N = case["P"], case["T"], case["N"]
    if case["op"] == "linear":
        K = case["K"]
        x = torch.empty((P, T, K), dtype=torch.bfloat16, device=dev)
        for p in range(P):
            x[p] = _widen(_normal(g, (T, K), dev, 0.5), g, dev, 8.0).to(torch.bfloat16)
        s["x"] = x
        s["out"] = torch.empty((P, T, N), dtype=DTYPES[case["y"]], device=dev)
        s["bias"] = _normal(g, (P, N), dev, 0.1) if case["bias"] else None
    else:
        K = case["H"]
        s["q"] = torch.empty((T, K), dtype=torch.int8, device=dev)
        s["q_scale"] = torch.empty((T,), dtype=torch.float32, device=dev)
        s["out"] = torch.empty((P, T, N), dtype=torch.bfloat16, device=dev)
        s["bias"] = None
    s["w"], s["w_scale"] = _weights(g, P, N, K, dev)
    return s


# ---- plain forms: elementary operations in 32 bits, rounded once at the end ----

def _plain_norm(v, kind, weight, bias):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(dim=-1, keepdim=True)
    v = v * torch.rsqrt((v * v).mean(dim=-1, keepdim=True) + NORM_EPS) * weight
    return v if bias is None else v + bias


def _plain_block(s):
    """(r', n) in fp32."""
    case = s["case"]
    T, H = s["y"].shape
    u = _plain_norm(s["y"].float(), case.get("post", "rms"), s["post_weight"], s["post_bias"])
    if s["gate"] is not None:
        G = s["gate"].shape[0]
        u = (u.view(G, T // G, H) * s["gate"].float().unsqueeze(1)).view(T, H)
    r = s["residual"].float() + case.get("alpha", 1.0) * u
    return r, _plain_norm(r, case.get("pre", "rms"), s["pre_weight"], s["pre_bias"])


def _plain_codes(x):
    """8-bit codes (as fp32) and the scale of each row; ties round away from zero."""
    m = x.abs().amax(dim=-1, keepdim=True)
    v = x * 127.0 / torch.where(m > 0, m, torch.ones_like(m))
    return torch.sign(v) * torch.floor(v.abs() + 0.5), m / torch.full_like(m, 127.0)


def _plain_product(codes, scale, s, dtype):
    """codes [P or 1,T,K], scale [P or 1,T,1]."""
    w = s["w"].float().transpose(1, 2)
    y = torch.matmul(codes, w) * scale * s["w_scale"].unsqueeze(1)
    if s["bias"] is not None:
        y = y + s["bias"].unsqueeze(1)
    return y.to(dtype)


def _run_plain(s):
    case = s["case"]
    if case["op"] == "norm":
        r, n = _plain_block(s)
        return r.to(DTYPES[case["residual"]]), n.to(DTYPES[case["n"]])
    if case["op"] == "linear":
        codes, scale = _plain_codes(s["x"].float())
        return _plain_product(codes, scale, s, DTYPES[case["y"]])
    r, n = _plain_block(s)
    codes, scale = _plain_codes(n)
    return r.to(DTYPES[case["residual"]]), _plain_product(codes, scale, s, torch.bfloat16)


# ---- the framework's calls ----------------------------------------------------

def _run_own(s):
    import bit_tensor_activation_amd as B
    case = s["case"]
    if case["op"] == "linear":
        return B.btq_int8_linear(s["x"], s["w"], s["w_scale"], bias=s["bias"], y=s["out"])
    if case["op"] == "norm":
        return B.btq_block_norm(
            s["y"], s["residual"], post=case["post"], post_weight=s["post_weight"],
            post_bias=s["post_bias"], gate=s["gate"], alpha=case["alpha"], pre=case["pre"],
            pre_weight=s["pre_weight"], pre_bias=s["pre_bias"], eps=NORM_EPS,
            residual_out=s["residual_out"], n=s["n"])
    r, q, q_scale = B.btq_block_norm(
        s["y"], s["residual"], post="rms", post_weight=s["post_weight"], pre="rms",
        pre_weight=s["pre_weight"], eps=NORM_EPS, residual_out=s["residual_out"], n=s["q"],
        n_scale=s["q_scale"])
    return r, B.btq_int8_matmul(q, q_scale, s["w"], s["w_scale"], y=s["out"])


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "linear":
        P, T, K, N = case["P"], case["T"], case["K"], case["N"]
        return {"bytes": P * (2 * T * K + N * K + 4 * N + size[case["y"]] * T * N
                              + (4 * N if case["bias"] else 0)),
                "flops": 2 * P * T * K * N}
    T, H = case["T"], case["H"]
    stream = T * H * (size[case["y"]] + 2 * size[case["residual"]])
    if case["op"] == "norm":
        per_feature = 4 * H * ({"none": 0, "rms": 1, "layer": 2}[case["post"]]
                               + {"none": 0, "rms": 1, "layer": 2}[case["pre"]])
        gate = 0 if case["gate"] == "none" else case["gate_rows"] * H * size[case["gate"]]
        return {"bytes": stream + T * H * size[case["n"]] + per_feature + gate,
                "flops": 12 * T * H}
    P, N = case["P"], case["N"]
    return {"bytes": stream + 8 * H + P * (N * H + 4 * N + 2 * T * N),
            "flops": 12 * T * H + 2 * P * T * H * N}


# ---- the definition in 64 bits --------------------------------------------------

def _rows64(v, kind, weight, bias):
    if kind == "none":
        return v
    d = v.shape[-1]
    if kind == "layer":
        v = v - v.sum(-1, keepdim=True) / d
    rms = ((v ** 2).sum(-1, keepdim=True) / d + NORM_EPS) ** 0.5
    out = v / rms * weight.double()
    return out if bias is None else out + bias.double()


def _block64(s):
    case = s["case"]
    u = _rows64(s["y"].double(), case.get("post", "rms"), s["post_weight"], s["post_bias"])
    if s["gate"] is not None:
        each = s["y"].shape[0] // s["gate"].shape[0]
        u = u * s["gate"].double().repeat_interleave(each, dim=0)
    r = s["residual"].double() + case.get("alpha", 1.0) * u
    return r, _rows64(r, case.get("pre", "rms"), s["pre_weight"], s["pre_bias"])


def _codes64(x):
    m = x.abs().max(-1, keepdim=True).values
    t = torch.where(m > 0, x * 127.0 / m.clamp_min(1e-300), torch.zeros_like(x))
    return torch.trunc(t + torch.copysign(torch.full_like(t, 0.5), t)), m / 127.0


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _block64(s)
    if case["op"] == "step":
        r, n = _block64(s)
        q, sc = _codes64(n)
    y = []
    for p in range(case["P"]):
        if case["op"] == "linear":
            q, sc = _codes64(s["x"][p].double())
        wt = s["w"][p].double().t().contiguous()
        v = q @ wt * sc * s["w_scale"][p].double()
        y.append(v if s["bias"] is None else v + s["bias"][p].double())
    y = torch.stack(y)
    return (r, y) if case["op"] == "step" else y
