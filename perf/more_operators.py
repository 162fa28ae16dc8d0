"""The measured cases of the attention between two linear layers: heads are
normed and rotated, keys and values go into a paged cache of 4-bit codes, and
queries attend over that cache.

Four paths, chosen by a case's "op":
  heads      btq_head_norm_rope: each query and key head is normed over its D
             features and rotated by its token's position.
  append     btq_kv_append of new keys (rotated on the way) and values to the
             cache, then btq_kv_gather of the values that it now holds for them.
  attention  btq_kv_attention of queries over the cached keys and values.
  step       rotation of the queries, append, attention, and the appended values.

Sizes are those of the codec's workloads (P shards, T tokens, H features) with
heads of 128 features, split over the shards: H=8192 is 64 query heads, 8 a
shard, H=4096 is 32. The ragged ones are generic.

The cache is uint8 [P,pages,Hkv,page/32,32*D+256]: for 32 tokens of a head,
keys [32][D/2] (feature 2i in the low nibble of byte i), values [D][16] (token
2i in the low nibble of byte i), then a word for each key and one for each
value: the scale's bf16 bits in the high half, those of 128+z in the low half.
A code c stands for scale*(c - z).
"""
from __future__ import annotations

import torch

own = False

EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
MAX_CACHE = 8 * 64 * 4096 * 128          # values of keys in a cache, largest listed decode
MAX_PAIRS = 8 * 8 * 2048 * 2048          # (query, key) pairs of all heads, listed prefill
MAX_ROWS = 8 * 8192 * 18 * 128           # values that the largest listed head norm takes


def _heads(name, P, T, Hq, Hk, D, rope_dim, norm="rms", rope="half", x="bf16", y="bf16"):
    case = dict(op="heads", P=P, T=T, Hq=Hq, Hk=Hk, D=D, rope_dim=rope_dim, norm=norm, rope=rope,
                x=x, y=y)
    return dict(case, name=name) if name else case


def _append(name, P, B, new, cached, Hk, D, page, rope_dim, rope="half", x="bf16", y="bf16"):
    case = dict(op="append", P=P, B=B, new_lo=new[0], new_hi=new[1], cached_lo=cached[0],
                cached_hi=cached[1], Hq=0, Hk=Hk, D=D, page=page, rope_dim=rope_dim, rope=rope,
                x=x, y=y)
    return dict(case, name=name) if name else case


def _attention(name, P, B, new, cached, Hq, Hk, D, page, window=0, causal=True, lse=False):
    case = dict(op="attention", P=P, B=B, new_lo=new[0], new_hi=new[1], cached_lo=cached[0],
                cached_hi=cached[1], Hq=Hq, Hk=Hk, D=D, page=page, window=window, causal=causal,
                lse=lse)
    return dict(case, name=name) if name else case


def _step(name, P, B, cached, Hq, Hk, D, page):
    case = dict(op="step", P=P, B=B, new_lo=1, new_hi=1, cached_lo=cached[0], cached_hi=cached[1],
                Hq=Hq, Hk=Hk, D=D, page=page, rope_dim=D, rope="half", x="bf16", y="bf16",
                window=0, causal=True, lse=False)
    return dict(case, name=name) if name else case


def listed():
    return [
        # one token of a decode, H=8192 over 8 shards: latency
        _heads("heads decode 1", 8, 1, 8, 1, 128, 128),
        # odd sizes, layer norm, neighbouring features rotated, a part of each head only, fp32 out
        _heads("heads ragged", 3, 333, 5, 2, 96, 64, norm="layer", rope="pairs", y="f32"),
        # a long prefill, H=8192 over 4 shards
        _heads("heads prefill 8192", 4, 8192, 16, 2, 128, 128),
        # one token for each of 64 sequences of a decode batch
        _append("append decode 64", 8, 64, (1, 1), (100, 4000), 1, 128, 64, 128),
        # odd pieces of sequences that start and end inside a page, small heads
        _append("append ragged", 3, 7, (1, 90), (0, 200), 2, 64, 32, 32, rope="pairs"),
        # a prefill of 8 prompts
        _append("append prefill 16384", 8, 8, (2048, 2048), (0, 0), 1, 128, 64, 128),
        # one token of a decode of moderate length: latency
        _attention("attention decode 1", 8, 1, (1, 1), (1000, 1000), 8, 1, 128, 64),
        # a decode batch of sequences of many lengths: the cache from HBM
        _attention("attention decode 64", 8, 64, (1, 1), (1000, 4095), 8, 1, 128, 64),
        # one token of a very long context, with the sums that merge it with others
        _attention("attention long", 8, 1, (1, 1), (131071, 131071), 8, 1, 128, 128, lse=True),
        # a few tokens a sequence to check a draft, odd heads, a sliding window
        _attention("attention ragged", 3, 9, (1, 7), (0, 900), 6, 2, 64, 32, window=200),
        # a prompt in one call, H=8192 over 8 shards: the matrix rate
        _attention("attention prefill 2048", 8, 1, (2048, 2048), (0, 0), 8, 1, 128, 64),
        # a decode batch through all of it
        _step("step decode 32", 8, 32, (500, 2000), 8, 1, 128, 64),
    ]


def _size(rng, lo, hi):
    """Log-uniform in [lo, hi]."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(("heads", "append", "attention", "attention", "step"))
    P = rng.choice((1, 2, 3, 4, 8))
    D = rng.choice((64, 96, 128, 128, 128, 256))
    Hk = rng.choice((1, 1, 2, 3, 4))
    rope_dim = rng.choice((D, D, D // 2))
    rope = rng.choice(("half", "half", "pairs"))
    if op == "heads":
        Hq = Hk * rng.choice((1, 2, 4, 5, 8))
        T = max(1, min(_size(rng, 1, 8192), MAX_ROWS // (P * (Hq + Hk) * D)))
        return _heads(None, P, T, Hq, Hk, D, rope_dim, rng.choice(("rms", "rms", "layer")), rope,
                      rng.choice(("bf16", "bf16", "f32")), rng.choice(("bf16", "bf16", "f32")))
    page = rng.choice((32, 64, 64, 128))
    B = _size(rng, 1, 64)
    if op == "append":
        new = _size(rng, 1, max(1, min(2048, 16384 * 8 // (P * Hk * B))))
        lo = rng.randint(1, new)
        cached = _size(rng, 1, 4000)
        return _append(None, P, B, (lo, new), (rng.randint(0, cached), cached), Hk, D, page,
                       rope_dim, rope, rng.choice(("bf16", "bf16", "f32")))
    Hq = Hk * rng.choice((1, 2, 4, 5, 8, 16))
    most = max(64, min(131072, MAX_CACHE // (P * B * Hk * D)))
    cached = _size(rng, 32, most - 32)
    lo = rng.randint(cached // 4, cached)
    if op == "step":
        return _step(None, P, B, (lo, cached), Hq, Hk, D, page)
    new = _size(rng, 1, max(1, min(2048, MAX_PAIRS // (P * B * Hq * (cached + 2048)))))
    if new < 8 and rng.random() < 0.5:
        new = 1
    cached = max(1, min(cached, MAX_CACHE // (P * B * Hk * D) - new))
    lo = min(lo, cached)
    return _attention(None, P, B, (rng.randint(1, new), new), (lo, cached), Hq, Hk, D, page,
                      window=rng.choice((0, 0, 0, _size(rng, 16, 4096))),
                      causal=rng.random() < 0.85, lse=rng.random() < 0.3)


# ---- inputs -----------------------------------------------------------------

def _spread(lo, hi, i):
    return lo + (i * 7919 + i * i * 31) % (hi - lo + 1)


def _lengths(case):
    """(new tokens, tokens in the cache with them) of each sequence."""
    new = [_spread(case["new_lo"], case["new_hi"], 3 * b + 1) for b in range(case["B"])]
    return new, [n + _spread(case["cached_lo"], case["cached_hi"], 5 * b + 2)
                 for b, n in enumerate(new)]


def _normal(g, shape, sigma=1.0):
    return torch.randn(shape, generator=g, device="cuda:0") * sigma


def _rope_table(rows, rope_dim):
    pos = torch.arange(rows, dtype=torch.float64, device="cuda:0")
    freq = 10000.0 ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64, device="cuda:0") / rope_dim)
    angle = pos[:, None] * freq
    return torch.cos(angle).float(), torch.sin(angle).float()


def _pack_pairs(codes):
    return (codes[..., 0::2] | codes[..., 1::2] << 4).contiguous()


def _quantized(x):
    """Codes (uint8) and the parameter words (4 bytes each) of rows x [...,D]."""
    codes, scale, z = _plain_codes(x)
    words = torch.stack(((z + 128.0).to(torch.bfloat16), scale.to(torch.bfloat16)), dim=-1)
    return codes.to(torch.uint8), words.view(torch.uint8)


def _filled_cache(g, P, pages, Hk, nb, D):
    """A cache whose every place holds a key and a value."""
    cache = torch.empty((P, pages, Hk, nb, 32 * D + 256), dtype=torch.uint8, device="cuda:0")
    wide = torch.ones((Hk, 1, 1, D), device="cuda:0")
    wide[..., torch.randint(0, D, (max(1, D // 32),), generator=g, device="cuda:0")] = 3.0
    step = max(1, (1 << 25) // (Hk * nb * 32 * D))
    for p in range(P):
        for a in range(0, pages, step):
            part = cache[p, a:a + step]
            shape = part.shape[:3] + (32, D)
            codes, words = _quantized(_normal(g, shape) * wide)
            part[..., :16 * D] = _pack_pairs(codes).flatten(-2)
            part[..., 32 * D:32 * D + 128] = words.flatten(-2)
            codes, words = _quantized(_normal(g, shape))
            part[..., 16 * D:32 * D] = _pack_pairs(codes.transpose(-1, -2)).flatten(-2)
            part[..., 32 * D + 128:] = words.flatten(-2)
    return cache


def _prepare_heads(case, g):
    P, T, Hq, Hk, D = (case[k] for k in ("P", "T", "Hq", "Hk", "D"))
    # the rows of a fused projection: queries, keys, values
    qkv = _normal(g, (P, T, Hq + 2 * Hk, D)).to(DTYPES[case["x"]])
    rows = max(4096, T)
    cos, sin = _rope_table(rows, case["rope_dim"])
    return {"case": case, "x": qkv[:, :, :Hq + Hk], "cos": cos, "sin": sin,
            "positions": torch.randint(0, rows, (T,), generator=g, device="cuda:0").int(),
            "q_weight": 1.0 + _normal(g, (D,), 0.1), "k_weight": 1.0 + _normal(g, (D,), 0.1),
            "y": torch.empty((P, T, Hq + Hk, D), dtype=DTYPES[case["y"]], device="cuda:0")}


def prepare(case, seed):
    g = torch.Generator(device="cuda:0")
    g.manual_seed(int(seed))
    if case["op"] == "heads":
        return _prepare_heads(case, g)
    P, B, Hq, Hk, D, page = (case[k] for k in ("P", "B", "Hq", "Hk", "D", "page"))
    new, lengths = _lengths(case)
    T = sum(new)
    each = -(-max(lengths) // page)
    held = [-(-n // page) for n in lengths]
    pages = sum(held) + 3
    order = torch.randperm(pages, generator=g, device="cuda:0").int()
    table = torch.full((B, each), -1, dtype=torch.int32, device="cuda:0")
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s = {"case": case, "table": table, "max_length": max(lengths), "max_new": max(new),
         "starts": torch.tensor(starts, dtype=torch.int32, device="cuda:0"),
         "lengths": torch.tensor(lengths, dtype=torch.int32, device="cuda:0")}
    if case["op"] == "append":
        s["cache"] = torch.zeros((P, pages, Hk, page // 32, 32 * D + 256), dtype=torch.uint8,
                                 device="cuda:0")
    else:
        s["cache"] = _filled_cache(g, P, pages, Hk, page // 32, D)
    if case["op"] != "attention":
        dt = DTYPES[case["x"]]
        qkv = _normal(g, (P, T, Hq + 2 * Hk, D))
        if case["op"] == "append":       # a few features are wide, the same ones for every token
            qkv[..., torch.randint(0, D, (D // 32,), generator=g, device="cuda:0")] *= 4.0
        qkv = qkv.to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], qkv[:, :, Hq + Hk:]
        s["cos"], s["sin"] = _rope_table(max(lengths), case["rope_dim"])
        s["k_out"] = torch.empty((P, T, Hk, D), dtype=DTYPES[case["y"]], device="cuda:0")
        s["v_out"] = torch.empty_like(s["k_out"])
    if case["op"] == "step":
        s["positions"] = (s["lengths"] - 1).contiguous()
        s["q_rot"] = torch.empty((P, T, Hq, D), dtype=torch.bfloat16, device="cuda:0")
    if case["op"] == "attention":
        s["q"] = _normal(g, (P, T, Hq, D), 1.5).to(torch.bfloat16)
    if case["op"] != "append":
        s["out"] = torch.empty((P, T, Hq * D), dtype=torch.bfloat16, device="cuda:0")
        s["lse"] = (torch.empty((P, T, Hq), dtype=torch.float32, device="cuda:0")
                    if case["lse"] else None)
    return s


# ---- plain forms: elementary operations in 32 bits, rounded once at the end ----

def _plain_rope(x, cos, sin, style):
    """x [...,D] by cos, sin [...,rope_dim/2]; the features past rope_dim stay."""
    r = 2 * cos.shape[-1]
    if style == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., r:]), dim=-1)
    a, b = x[..., 0:r:2], x[..., 1:r:2]
    pairs = torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2)
    return torch.cat((pairs, x[..., r:]), dim=-1)


def _plain_heads(s):
    case = s["case"]
    x = s["x"].float()
    if case["norm"] == "layer":
        x = x - x.mean(dim=-1, keepdim=True)
    x = x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS)
    x = torch.cat((x[:, :, :case["Hq"]] * s["q_weight"], x[:, :, case["Hq"]:] * s["k_weight"]), 2)
    at = s["positions"].long()
    y = _plain_rope(x, s["cos"][at].unsqueeze(1), s["sin"][at].unsqueeze(1), case["rope"])
    return y.to(DTYPES[case["y"]])


def _plain_codes(x):
    """Codes, scale and z of rows x [...,D]: scale is the range (0 in it) over 15,
    rounded up to bf16; everything is held in 32 bits."""
    lo = x.amin(dim=-1, keepdim=True).clamp_max(0.0)
    hi = x.amax(dim=-1, keepdim=True).clamp_min(0.0)
    scale = (hi - lo) / torch.full_like(hi, 15.0)
    scale = ((scale.view(torch.int32) + 0xffff) & -65536).view(torch.float32)
    scale = torch.where(scale < 2.0 ** -126, torch.ones_like(scale), scale)
    z = torch.round(-lo / scale).clamp(0.0, 15.0)
    return (torch.round(x / scale) + z).clamp(0.0, 15.0), scale.squeeze(-1), z.squeeze(-1)


def _plain_rows(s):
    """(sequence, place in it) of each token."""
    T = s["out"].shape[1] if "out" in s else s["k"].shape[1]
    rows = torch.arange(T, device="cuda:0", dtype=torch.int32)
    seq = torch.searchsorted(s["starts"][1:].contiguous(), rows, right=True)
    new = s["starts"][1:] - s["starts"][:-1]
    return seq, (rows - s["starts"][seq] + s["lengths"][seq] - new[seq]).long()


def _plain_held(x):
    """What the cache holds for rows x: scale*(code - z)."""
    codes, scale, z = _plain_codes(x)
    return (codes - z.unsqueeze(-1)) * scale.unsqueeze(-1)


def _plain_append(s):
    """The appended keys and values as the cache holds them, in fp32."""
    _, place = _plain_rows(s)
    cos, sin = s["cos"][place].unsqueeze(1), s["sin"][place].unsqueeze(1)
    return (_plain_held(_plain_rope(s["k"].float(), cos, sin, s["case"]["rope"])),
            _plain_held(s["v"].float()))


def _plain_unpack(s):
    """All sequences' keys and values, [P,B,Hk,L,D] in fp32, L the longest rounded
    up to pages. Places without a page hold those of page 0."""
    D = s["case"]["D"]
    r = s["cache"][:, s["table"].clamp_min(0).long()].permute(0, 1, 3, 2, 4, 5).flatten(3, 4)

    def value(code, words):
        w = words.contiguous().view(torch.bfloat16).view(words.shape[:-1] + (32, 2)).float()
        return ((code.float() - (w[..., :1] - 128.0)) * w[..., 1:]).flatten(3, 4)
    k = r[..., :16 * D].unflatten(-1, (32, D // 2))
    k = torch.stack((k & 15, k >> 4), dim=-1).flatten(-2)
    v = r[..., 16 * D:32 * D].unflatten(-1, (D, 16))
    v = torch.stack((v & 15, v >> 4), dim=-1).flatten(-2).transpose(-1, -2)
    return (value(k, r[..., 32 * D:32 * D + 128]), value(v, r[..., 32 * D + 128:]))


def _plain_attention(s, q, k, v):
    case = s["case"]
    P, B, Hq, Hk, D = (case[c] for c in ("P", "B", "Hq", "Hk", "D"))
    N, L, G = s["max_new"], k.shape[3], Hq // Hk
    new = (s["starts"][1:] - s["starts"][:-1]).long()
    i = torch.arange(N, device="cuda:0")
    rows = s["starts"][:-1, None].long() + torch.minimum(i, new[:, None] - 1)      # [B,N]
    qb = q[:, rows].float().view(P, B, N, Hk, G, D).permute(0, 1, 3, 2, 4, 5)
    scores = torch.matmul(qb.reshape(P, B, Hk, N * G, D), k.transpose(-1, -2)) * D ** -0.5
    place = (s["lengths"].long() - new)[:, None] + i                               # [B,N]
    key = torch.arange(L, device="cuda:0")
    seen = (key < s["lengths"][:, None, None]).expand(B, N, L)
    if case["causal"]:
        seen = seen & (key <= place[..., None])
    if case["window"]:
        seen = seen & (key > place[..., None] - case["window"])
    seen = seen.unsqueeze(2).expand(B, N, G, L).reshape(1, B, 1, N * G, L)
    scores = scores.masked_fill(~seen, float("-inf"))
    top = scores.amax(dim=-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    e = torch.exp(scores - top)
    total = e.sum(dim=-1, keepdim=True)
    o = torch.matmul(e, v) / torch.where(total > 0, total, torch.ones_like(total))

    def by_token(t, width):      # [P,B,Hk,N*G,width] -> [P,T,Hq*width]
        seq, at = _plain_rows(s)
        t = t.view(P, B, Hk, N, G, width).permute(0, 1, 3, 2, 4, 5)
        return t[:, seq, at - (s["lengths"].long() - new)[seq]].reshape(P, -1, Hq * width)
    out = by_token(o, D).to(torch.bfloat16)
    return (out, by_token(top + torch.log(total), 1)) if case["lse"] else (out,)


def _plain_step(s):
    at = s["positions"].long()
    q = _plain_rope(s["q"].float(), s["cos"][at].unsqueeze(1), s["sin"][at].unsqueeze(1), "half")
    new_k, new_v = _plain_append(s)
    k, v = _plain_unpack(s)
    seq = torch.arange(s["case"]["B"], device="cuda:0")
    k[:, seq, :, at] = new_k.transpose(0, 1)
    v[:, seq, :, at] = new_v.transpose(0, 1)
    out, = _plain_attention(s, q.to(torch.bfloat16), k, v)
    return out, new_k.to(torch.bfloat16), new_v.to(torch.bfloat16)


def _run_plain(s):
    case = s["case"]
    if case["op"] == "heads":
        return _plain_heads(s)
    if case["op"] == "append":
        k, v = _plain_append(s)
        return k.to(DTYPES[case["y"]]), v.to(DTYPES[case["y"]])
    if case["op"] == "step":
        return _plain_step(s)
    return _plain_attention(s, s["q"], *_plain_unpack(s))


# ---- the framework's calls ----------------------------------------------------

def _own_append(s):
    import bit_tensor_activation_amd as B
    B.btq_kv_append(s["k"], s["v"], s["starts"], s["lengths"], s["table"], s["cache"],
                    cos=s["cos"], sin=s["sin"], rope=s["case"]["rope"])
    return B.btq_kv_gather(s["starts"], s["lengths"], s["table"], s["cache"], k=s["k_out"],
                           v=s["v_out"])


def _own_attention(s, q):
    import bit_tensor_activation_amd as B
    return B.btq_kv_attention(q, s["starts"], s["lengths"], s["table"], s["cache"],
                              causal=s["case"]["causal"], window=s["case"]["window"],
                              max_length=s["max_length"], out=s["out"], lse=s["lse"])


def _run_own(s):
    import bit_tensor_activation_amd as B
    case = s["case"]
    if case["op"] == "heads":
        return B.btq_head_norm_rope(s["x"], case["Hq"], norm=case["norm"], q_weight=s["q_weight"],
                                    k_weight=s["k_weight"], eps=EPS, positions=s["positions"],
                                    cos=s["cos"], sin=s["sin"], rope=case["rope"], out=s["y"])
    if case["op"] == "append":
        return _own_append(s)
    if case["op"] == "attention":
        out = _own_attention(s, s["q"])
        return (out, s["lse"]) if case["lse"] else (out,)
    B.btq_head_norm_rope(s["q"], case["Hq"], norm="none", positions=s["positions"], cos=s["cos"],
                         sin=s["sin"], out=s["q_rot"])
    k, v = _own_append(s)
    return _own_attention(s, s["q_rot"]), k, v


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    size = {"f32": 4, "bf16": 2}
    P, Hq, Hk, D = (case[k] for k in ("P", "Hq", "Hk", "D"))
    if case["op"] == "heads":
        T, n = case["T"], P * case["T"] * (Hq + Hk) * D
        return {"bytes": n * (size[case["x"]] + size[case["y"]]) + T * 4 * (case["rope_dim"] + 1)
                + 8 * D, "flops": 8 * n}
    new, lengths = _lengths(case)
    T, B = sum(new), case["B"]
    row = P * Hk * (D + 8)                       # a token's codes and words, keys and values
    found = {"bytes": 0, "flops": 0}
    if case["op"] != "attention":
        n = 2 * P * T * Hk * D
        found["bytes"] += (n * (size[case["x"]] + size[case["y"]]) + T * row
                           + 4 * T * case["rope_dim"])
        found["flops"] += 10 * n
    if case["op"] != "append":
        places = pairs = 0
        for n, length in zip(new, lengths):
            first = length - n
            if case["window"]:
                seen = [min(p + 1 if case["causal"] else length, length)
                        - max(0, p + 1 - case["window"]) for p in range(first, length)]
                places += length - max(0, first + 1 - case["window"])
                pairs += sum(seen)
            else:
                places += length
                pairs += (n * first + n * (n + 1) // 2) if case["causal"] else n * length
        found["bytes"] += places * row + P * T * Hq * D * 4 + 4 * B * 2
        if case["lse"]:
            found["bytes"] += 4 * P * T * Hq
        found["flops"] += 4 * D * P * Hq * pairs
    return found


# ---- the definition in 64 bits --------------------------------------------------

def _turn64(x, cos, sin, style):
    """Rotation as a product of complex numbers."""
    n = cos.shape[-1]
    at = torch.arange(n, device=x.device)
    i, j = (at, at + n) if style == "half" else (2 * at, 2 * at + 1)
    w = torch.complex(x[..., i], x[..., j]) * torch.complex(cos.double(), sin.double())
    y = x.clone()
    y[..., i], y[..., j] = w.real, w.imag
    return y


def _held64(x):
    low = torch.minimum(x.min(-1).values, torch.zeros((), dtype=x.dtype, device=x.device))
    high = torch.maximum(x.max(-1).values, torch.zeros((), dtype=x.dtype, device=x.device))
    m, e = torch.frexp((high - low) / 15)
    step = torch.ldexp(torch.ceil(m * 256) / 256, e)
    step = torch.where(step < 2.0 ** -126, torch.ones_like(step), step)[..., None]
    zero = torch.round(-low[..., None] / step)
    return ((torch.round(x / step) + zero).clamp(0, 15) - zero) * step


def _appended64(s):
    starts, lengths = s["starts"].tolist(), s["lengths"].tolist()
    place = torch.cat([torch.arange(n - (b - a), n, device="cuda:0")
                       for a, b, n in zip(starts, starts[1:], lengths)])
    k = _turn64(s["k"].double(), s["cos"][place][:, None], s["sin"][place][:, None],
                s["case"]["rope"])
    return _held64(k), _held64(s["v"].double())


def _sequence64(s, b, length):
    """Keys and values [P,Hk,length,D] of one sequence, by its places one page after another."""
    D, page = s["case"]["D"], s["case"]["page"]
    t = torch.arange(length, device="cuda:0")
    r = s["cache"][:, s["table"][b, t // page].long(), :, t % page // 32]       # [n,P,Hk,bytes]
    r = r.permute(1, 2, 0, 3)
    i = t % 32
    d = torch.arange(D, device="cuda:0")
    kb = r[:, :, t[:, None], (i * (D // 2))[:, None] + d // 2].int()
    kc = torch.where(d % 2 == 1, kb // 16, kb % 16)
    vb = r[:, :, t[:, None], 16 * D + d * 16 + (i // 2)[:, None]].int()
    vc = torch.where((i % 2 == 1)[:, None], vb // 16, vb % 16)

    def held(c, first):
        w = r[:, :, t[:, None], first + 4 * i[:, None] + torch.arange(4, device="cuda:0")].int()
        step = ((w[..., 2] << 16) | (w[..., 3] << 24)).view(torch.float32).double()
        zero = ((w[..., 0] << 16) | (w[..., 1] << 24)).view(torch.float32).double() - 128
        return (c.double() - zero[..., None]) * step[..., None]
    return held(kc, 32 * D), held(vc, 32 * D + 128)


def _attention64(s, q, new=None):
    case = s["case"]
    G, D = case["Hq"] // case["Hk"], case["D"]
    starts, lengths = s["starts"].tolist(), s["lengths"].tolist()
    outs, sums = [], []
    for b, length in enumerate(lengths):
        n = starts[b + 1] - starts[b]
        k, v = _sequence64(s, b, length)
        if new is not None:
            k[:, :, length - n:] = new[0][:, starts[b]:starts[b + 1]].transpose(1, 2)
            v[:, :, length - n:] = new[1][:, starts[b]:starts[b + 1]].transpose(1, 2)
        at = torch.arange(length - n, length, device="cuda:0")[:, None]
        key = torch.arange(length, device="cuda:0")
        hidden = torch.zeros((n, length), dtype=torch.bool, device="cuda:0")
        if case["causal"]:
            hidden |= key > at
        if case["window"]:
            hidden |= key <= at - case["window"]
        o, l = [], []
        for h in range(case["Hq"]):
            x = q[:, starts[b]:starts[b + 1], h].double()
            a = torch.bmm(x, k[:, h // G].transpose(1, 2).contiguous()) / D ** 0.5
            a[:, hidden] = -float("inf")
            total = torch.logsumexp(a, -1)
            p = torch.where(hidden.all(-1)[:, None], torch.zeros_like(a),
                            torch.exp(a - total[..., None]))
            o.append(torch.bmm(p, v[:, h // G].contiguous()))
            l.append(total)
        outs.append(torch.cat(o, -1))
        sums.append(torch.stack(l, -1))
    out = torch.cat(outs, 1)
    return (out, torch.cat(sums, 1)) if case["lse"] else (out,)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "heads":
        x = s["x"].double()
        if case["norm"] == "layer":
            x = x - x.sum(-1, keepdim=True) / case["D"]
        x = x / ((x ** 2).sum(-1, keepdim=True) / case["D"] + EPS) ** 0.5
        x[:, :, :case["Hq"]] *= s["q_weight"].double()
        x[:, :, case["Hq"]:] *= s["k_weight"].double()
        at = s["positions"].long()
        return _turn64(x, s["cos"][at][:, None], s["sin"][at][:, None], case["rope"])
    if case["op"] == "append":
        return _appended64(s)
    if case["op"] == "attention":
        return _attention64(s, s["q"])
    at = s["positions"].long()
    q = _turn64(s["q"].double(), s["cos"][at][:, None], s["sin"][at][:, None], "half")
    new = _appended64(s)
    return _attention64(s, q, new) + new
