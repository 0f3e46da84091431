"""Cases of the operators around a mixture-of-experts block: the norm between
blocks, the routing of tokens to experts, and the expert layer on FP4 and FP8
weights.

A case is a dict of plain values.  ``run`` computes it in plain torch (32 bits,
64 where a comparison hangs on the last bits) or, where ``own`` is set, with
this repository's library; ``exact`` computes it in 64 bits from the
definition.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # closes a block and opens the next for one token that is being decoded
        {"name": "norm_token", "op": "norm", "M": 1, "K": 5120, "dtype": "bf16", "post": True, "pre": True,
         "gate": "none", "residual": True, "scale": 1.0, "offset": 0.0},
        # a decode batch of odd size in rows of odd length, with a gate for every value
        {"name": "norm_batch_odd", "op": "norm", "M": 77, "K": 2049, "dtype": "fp16", "post": True, "pre": True,
         "gate": "full", "residual": True, "scale": 0.5, "offset": 1.0},
        # a prompt: the plain "add to the residual, then norm" of most models
        {"name": "norm_prompt", "op": "norm", "M": 8192, "K": 5120, "dtype": "bf16", "post": False, "pre": True,
         "gate": "row", "residual": True, "scale": 0.22, "offset": 0.0},
        # routing of one token
        {"name": "route_token", "op": "route", "M": 1, "E": 128, "topk": 8, "dtype": "fp32", "score": "softmax",
         "bias": False, "renormalize": True, "scale": 1.0},
        # routing of a prompt, with sigmoid scores and a selection bias that balances the experts
        {"name": "route_prompt", "op": "route", "M": 8192, "E": 256, "topk": 8, "dtype": "bf16", "score": "sigmoid",
         "bias": True, "renormalize": True, "scale": 2.5},
        # one token, many small experts: 8 of them are read, launch and latency count
        {"name": "fp4_moe_token", "op": "moe", "format": "fp4", "M": 1, "E": 128, "topk": 8, "K": 2048, "I": 768,
         "dtype": "bf16", "act": "silu", "local": 1.0},
        # four tokens (or one with drafted ones) on large experts
        {"name": "fp4_moe_wide", "op": "moe", "format": "fp4", "M": 4, "E": 64, "topk": 8, "K": 7168, "I": 2048,
         "dtype": "bf16", "act": "silu", "local": 1.0},
        # a decode batch: most experts are read, by one to six tokens each
        {"name": "fp4_moe_batch", "op": "moe", "format": "fp4", "M": 32, "E": 128, "topk": 8, "K": 2048, "I": 768,
         "dtype": "fp16", "act": "silu", "local": 1.0},
        # a large batch on few experts with sizes that end inside a tile: about 16 tokens for each
        {"name": "fp4_moe_128", "op": "moe", "format": "fp4", "M": 128, "E": 32, "topk": 4, "K": 2880, "I": 2880,
         "dtype": "bf16", "act": "gelu", "local": 1.0},
        # one token on FP8 experts
        {"name": "fp8_moe_token", "op": "moe", "format": "fp8", "M": 1, "E": 64, "topk": 6, "K": 2048, "I": 1408,
         "dtype": "bf16", "act": "silu", "local": 1.0},
        # a decode batch on FP8 experts
        {"name": "fp8_moe_batch", "op": "moe", "format": "fp8", "M": 16, "E": 128, "topk": 8, "K": 4096, "I": 1024,
         "dtype": "bf16", "act": "silu", "local": 1.0},
        # expert parallelism: this device holds a quarter of the experts, the other choices are masked
        {"name": "fp8_moe_shard", "op": "moe", "format": "fp8", "M": 100, "E": 16, "topk": 6, "K": 5120, "I": 1280,
         "dtype": "fp16", "act": "silu", "local": 0.25},
    ]


MOST_READ = {"fp4": 1.15e9, "fp8": 1.65e9}  # weights that one pass reads, at most (the largest listed cases)
MOST_HELD = 2.9e9  # weights of all experts, at most


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("norm", "route", "fp4", "fp8"))
    if kind == "norm":
        step = rng.choice((1, 8, 64))
        return {"op": "norm", "M": _log(rng, 1, 8192), "K": _log(rng, 64, 5120) // step * step,
                "dtype": rng.choice(("bf16", "fp16")), "post": rng.random() < 0.5, "pre": rng.random() < 0.8,
                "gate": rng.choice(("none", "row", "full")), "residual": rng.random() < 0.8,
                "scale": rng.choice((1.0, 0.5, 0.22)), "offset": rng.choice((0.0, 1.0))}
    if kind == "route":
        E = _log(rng, 8, 512)
        return {"op": "route", "M": _log(rng, 1, 8192), "E": E, "topk": rng.randint(1, min(8, E)),
                "dtype": rng.choice(("fp32", "bf16", "fp16")), "score": rng.choice(("softmax", "sigmoid")),
                "bias": rng.random() < 0.4, "renormalize": rng.random() < 0.7, "scale": rng.choice((1.0, 2.5))}
    while True:
        c = {"op": "moe", "format": kind, "M": _log(rng, 1, 128), "E": _log(rng, 8, 256), "topk": rng.randint(1, 8),
             "K": 64 * _log(rng, 8, 112), "I": 64 * _log(rng, 6, 45), "dtype": rng.choice(("bf16", "fp16")),
             "act": rng.choice(("silu", "silu", "gelu")), "local": rng.choice((1.0, 1.0, 0.25))}
        one = 3.0 * c["K"] * c["I"]
        if one * min(c["M"] * c["topk"], c["E"]) <= MOST_READ[kind] and one * c["E"] <= MOST_HELD:
            return c


# ------------------------------------------------------------------ inputs

def _e4m3(shape, lo, hi, g):
    return torch.empty(shape, device="cuda").uniform_(lo, hi, generator=g).to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    normal = lambda *shape: torch.empty(shape, device="cuda").normal_(generator=g)  # noqa: E731
    M = case["M"]
    s = {"case": case}
    if case["op"] == "norm":
        K = case["K"]
        s["x"] = normal(M, K).mul_(0.7).to(dt)
        s["residual"] = normal(M, K).mul_(3.0).to(dt) if case["residual"] else None
        weight = lambda: (1.0 - case["offset"] + 0.2 * normal(K)).to(dt)  # noqa: E731
        s["post"] = weight() if case["post"] else None
        s["pre"] = weight() if case["pre"] else None
        s["gate"] = None if case["gate"] == "none" else normal(*((K,) if case["gate"] == "row" else (M, K))).sigmoid_().to(dt)
        return s
    if case["op"] == "route":
        s["logits"] = normal(M, case["E"]).mul_(1.5).to(dt)
        s["bias"] = normal(case["E"]).mul_(0.1) if case["bias"] else None
        return s
    E, K, inner, topk, fp4 = case["E"], case["K"], case["I"], case["topk"], case["format"] == "fp4"
    s["A"] = normal(M, K).to(dt)
    # a token's experts: the best of all, those of other devices masked by -1
    everywhere = max(topk, int(round(E / case["local"])))
    score, ids = (normal(M, everywhere) + 0.5 * normal(everywhere)).topk(topk, dim=1)
    s["ids"] = torch.where(ids < E, ids, -1).to(torch.int32)
    s["weights"] = score.softmax(1)
    if fp4:
        s["w13"] = torch.randint(0, 256, (E, 2 * inner, K // 2), dtype=torch.uint8, device="cuda", generator=g)
        s["w2"] = torch.randint(0, 256, (E, K, inner // 2), dtype=torch.uint8, device="cuda", generator=g)
        s["s13"] = _e4m3((E, 2 * inner, K // 16), 0.5, 4.0, g)
        s["s2"] = _e4m3((E, K, inner // 16), 0.5, 4.0, g)
        s["g13"] = torch.empty(E, device="cuda").uniform_(0.1, 0.18, generator=g) / math.sqrt(K)
        s["g2"] = torch.empty(E, device="cuda").uniform_(0.1, 0.18, generator=g) / math.sqrt(inner)
    else:
        # every finite E4M3 code
        def codes(*shape):
            w = torch.randint(0, 254, shape, dtype=torch.uint8, device="cuda", generator=g)
            return w.add_(w >= 127)
        s["w13"], s["w2"] = codes(E, 2 * inner, K), codes(E, K, inner)
        cols = lambda n: (n + 127) // 128  # noqa: E731
        s["s13"] = torch.empty(E, 2 * inner, cols(K), device="cuda").uniform_(0.005, 0.01, generator=g) / math.sqrt(K)
        s["s2"] = torch.empty(E, K, cols(inner), device="cuda").uniform_(0.005, 0.01, generator=g) / math.sqrt(inner)
    return s


# ------------------------------------------------------------------ one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "route": _own_route, "moe": _own_moe}[op](state)
    return {"norm": _plain_norm, "route": _plain_route, "moe": _plain_moe}[op](state)


def _own_norm(s):
    import fp8_weight_only_fp4w_amd as fw
    c = s["case"]
    r, y = fw.fp4w_block_norm(s["x"], residual=s["residual"], pre_weight=s["pre"], post_weight=s["post"], gate=s["gate"],
                              scale=c["scale"], eps=1e-6, weight_offset=c["offset"])
    return {"residual": r, "y": y}


def _own_route(s):
    import fp8_weight_only_fp4w_amd as fw
    c = s["case"]
    ids, weights = fw.fp4w_moe_route(s["logits"], c["topk"], score=c["score"], select_bias=s["bias"],
                                     renormalize=c["renormalize"], scale=c["scale"])
    return {"ids": ids, "weights": weights}


def _own_moe(s):
    import fp8_weight_only_fp4w_amd as fw
    c = s["case"]
    if c["format"] == "fp4":
        return fw.fp4w_moe(s["A"], s["ids"], s["weights"], s["w13"], s["s13"], s["g13"], s["w2"], s["s2"], s["g2"],
                           block_size=16, activation=c["act"])
    return fw.fp8w_moe(s["A"], s["ids"], s["weights"], s["w13"], s["s13"], s["w2"], s["s2"], block_size=128,
                       activation=c["act"])


def _rms(x, weight, offset):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * (weight.float() + offset)


def _plain_norm(s):
    c, dt = s["case"], s["x"].dtype
    r = s["x"].float()
    if c["post"]:
        r = _rms(r, s["post"], c["offset"])
    if s["gate"] is not None:
        r = r * s["gate"].float()
    r = r * c["scale"]
    if c["residual"]:
        r = r + s["residual"].float()
    return {"residual": r.to(dt), "y": _rms(r, s["pre"], c["offset"]).to(dt) if c["pre"] else None}


def _plain_route(s):
    c = s["case"]
    x = s["logits"].double()  # the choice hangs on the last bits of a score with its bias
    score = x.softmax(-1) if c["score"] == "softmax" else x.sigmoid()
    key = x if s["bias"] is None else score + s["bias"].double()
    ids = key.sort(dim=-1, descending=True, stable=True).indices[:, : c["topk"]]  # stable: ties go to the lowest index
    w = score.gather(1, ids)
    if c["renormalize"]:
        w = w / w.sum(-1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": (w * c["scale"]).float()}


def _dequant(w, scale, second, fp4):
    """The weights of some experts in 32 bits."""
    if fp4:
        lut = torch.tensor(E2M1, device=w.device)
        v = lut[torch.stack((w & 15, w >> 4), -1).flatten(-2).int()]
        blocks = v.unflatten(-1, (-1, 16))
        blocks.mul_(scale.view(torch.float8_e4m3fn).float().unsqueeze(-1) * second.view(-1, 1, 1, 1))
        return v
    v = w.view(torch.float8_e4m3fn).float()
    return v.mul_(scale.repeat_interleave(128, -1)[..., : v.shape[-1]])


def _act(kind, x):
    if kind == "silu":
        return x / (1 + torch.exp(-x))
    return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))


def _plain_moe(s):
    c = s["case"]
    fp4, M, E, inner = c["format"] == "fp4", c["M"], c["E"], c["I"]
    A, mask = s["A"].float(), s["ids"] >= 0
    ids = torch.where(mask, s["ids"], 0).long()
    flat = ids.flatten()
    few = flat.numel() < E  # few choices: only their experts are expanded; else every expert, for every token
    of = lambda t: None if t is None else t[flat] if few else t  # noqa: E731
    h = _dequant(of(s["w13"]), of(s["s13"]), of(s.get("g13")), fp4)
    if few:
        h = torch.bmm(h, A.repeat_interleave(c["topk"], 0).unsqueeze(-1)).squeeze(-1)
    else:
        h = torch.matmul(A, h.transpose(1, 2))
    h = _act(c["act"], h[..., :inner]) * h[..., inner:]
    w2 = _dequant(of(s["w2"]), of(s["s2"]), of(s.get("g2")), fp4)
    if few:
        y = torch.bmm(w2, h.unsqueeze(-1)).view(M, c["topk"], -1)
    else:
        y = torch.matmul(h, w2.transpose(1, 2))[ids, torch.arange(M, device=ids.device).unsqueeze(-1)]
    return (y * (s["weights"] * mask).unsqueeze(-1)).sum(1).to(s["A"].dtype)


# ------------------------------------------------------------------ what it costs, and what it is

def _experts(case):
    """How many of the held experts a pass reads, on average over routings without favourites."""
    everywhere = max(case["topk"], int(round(case["E"] / case["local"])))
    return case["E"] * (1 - (1 - case["topk"] / everywhere) ** case["M"])


def work(case):
    M = case["M"]
    if case["op"] == "norm":
        K = case["K"]
        values = M * K * (2 + case["residual"] + case["pre"] + (case["gate"] == "full"))
        values += K * (case["pre"] + case["post"] + (case["gate"] == "row"))
        return {"bytes": 2 * values, "flops": M * K * (4 * (case["pre"] + case["post"]) + 3)}
    if case["op"] == "route":
        each = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": M * case["E"] * each + M * case["topk"] * 8 + 4 * case["E"] * case["bias"], "flops": M * case["E"] * 12}
    K, inner = case["K"], case["I"]
    if case["format"] == "fp4":
        expert = 3 * K * inner * 9 / 16 + 8
    else:
        expert = 3 * K * inner + 4 * (2 * inner * -(-K // 128) + K * -(-inner // 128))
    chosen = M * case["topk"] * case["local"]
    return {"bytes": _experts(case) * expert + 4 * M * K + 8 * M * case["topk"], "flops": 6 * chosen * K * inner}


def exact(case, seed):
    s = prepare(case, seed)
    up = lambda t: t.to(torch.float64)  # noqa: E731
    if case["op"] == "norm":
        norm = lambda v, w: v / (v.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * (up(w) + case["offset"])  # noqa: E731
        b = up(s["x"]) if s["post"] is None else norm(up(s["x"]), s["post"])
        r = case["scale"] * b * (1.0 if s["gate"] is None else up(s["gate"])) + (0.0 if s["residual"] is None else up(s["residual"]))
        return {"residual": r, "y": None if s["pre"] is None else norm(r, s["pre"])}
    if case["op"] == "route":
        x = up(s["logits"])
        if case["score"] == "softmax":
            p = torch.exp(x - x.amax(1, keepdim=True))
            p = p / p.sum(1, keepdim=True)
        else:
            p = 1 / (1 + torch.exp(-x))
        left = x.clone() if s["bias"] is None else p + up(s["bias"])
        ids, w = [], []
        for _ in range(case["topk"]):
            best = (left == left.amax(1, keepdim=True)).to(torch.int8).argmax(1, keepdim=True)  # the first of the largest
            ids.append(best)
            w.append(p.gather(1, best))
            left.scatter_(1, best, -math.inf)
        w = torch.cat(w, 1)
        if case["renormalize"]:
            w = w / w.sum(1, keepdim=True)
        return {"ids": torch.cat(ids, 1).to(torch.int32), "weights": w * case["scale"]}
    A, K, inner = up(s["A"]), case["K"], case["I"]
    y = torch.zeros(case["M"], K, dtype=torch.float64, device=A.device)

    def matrix(name, e):
        w, scale = s["w" + name][e], s["s" + name][e]
        if case["format"] == "fp8":
            return up(w.view(torch.float8_e4m3fn)) * torch.repeat_interleave(up(scale), 128, 1)[:, : w.shape[1]]
        v = torch.empty(w.shape[0], 2 * w.shape[1], dtype=torch.float64, device=w.device)
        for half, code in ((0, w % 16), (1, w // 16)):
            code = code.to(torch.int64)
            m, x = code % 2, code % 8 // 2  # E2M1: one bit of mantissa, two of exponent with bias 1
            v[:, half::2] = torch.where(code >= 8, -1.0, 1.0) * torch.where(x == 0, 0.5 * m, (1 + 0.5 * m) * 2.0 ** (x - 1))
        return v * torch.repeat_interleave(up(scale.view(torch.float8_e4m3fn)), 16, 1) * up(s["g" + name][e])

    for e in sorted(set(s["ids"].flatten().tolist()) - {-1}):
        weight = (up(s["weights"]) * (s["ids"] == e)).sum(1)
        rows = weight.nonzero().flatten()
        gate, value = (A[rows] @ matrix("13", e).T).split(inner, 1)
        if case["act"] == "silu":
            h = gate * torch.sigmoid(gate) * value
        else:
            h = 0.5 * gate * (1 + torch.tanh((2 / math.pi) ** 0.5 * (gate + 0.044715 * gate ** 3))) * value
        y[rows] += weight[rows, None] * (h @ matrix("2", e).T)
    return y
