"""Cases of the head's operators, from hidden rows to the log probabilities of tokens: the microscaled 4-bit format
(``mxfp4_quant``, ``mxfp4_dequant``), products of 4-bit operands (``mxfp4_linear_bf16``) and log probabilities of given
tokens with entropy and top alternatives (``m2_token_logprobs``).

With ``own`` false ``run`` computes them in plain torch; with ``own`` true it calls the package."""
import math

import torch

own = False


def listed():
    quant = {"op": "quant"}
    linear = {"op": "linear"}
    lp = {"op": "logprobs"}
    return [
        # one decode row to 4 bits and back: latency alone
        {"name": "quant_1", **quant, "rows": 1, "k": 2688, "pad": 0},
        # an odd number of rows that are a slice of wider ones (the z columns of in_proj's rows)
        {"name": "quant_1337_slice", **quant, "rows": 1337, "k": 4096, "pad": 6208},
        # the rows of the 4 x 2048 prefill: the bytes decide
        {"name": "quant_8192", **quant, "rows": 8192, "k": 2688, "pad": 0},
        # one row through a projection of the block's size: latency and one read of the weights
        {"name": "linear_1", **linear, "rows": 1, "k": 2688, "n": 10304, "out": "bf16"},
        # the 64-row decode batch, out_proj's size
        {"name": "linear_64", **linear, "rows": 64, "k": 4096, "n": 2688, "out": "bf16"},
        # odd sizes throughout: a chunk of a ragged prefill against a small head, f32 logits
        {"name": "linear_517_odd", **linear, "rows": 517, "k": 1056, "n": 5003, "out": "f32"},
        # the 4 x 2048 prefill through a projection of in_proj's size
        {"name": "linear_8192", **linear, "rows": 8192, "k": 2688, "n": 10304, "out": "bf16"},
        # the head of a decode batch over a large vocabulary: one read of the weights decides
        {"name": "head_64", **linear, "rows": 64, "k": 2688, "n": 131072, "out": "f32"},
        # one row of one request, twenty alternatives: latency alone
        {"name": "logprobs_1", **lp, "rows": 1, "vocab": 131072, "dtype": "bf16", "pad": 0, "top": 20, "masked": 0.0,
         "without": 0},
        # a decode batch, f32 logits, five alternatives
        {"name": "logprobs_64_f32", **lp, "rows": 64, "vocab": 65536, "dtype": "f32", "pad": 0, "top": 5, "masked": 0.0,
         "without": 0},
        # a ragged batch of prompts: odd vocabulary in padded rows, banned tokens, rows without a token to score
        {"name": "logprobs_333_odd", **lp, "rows": 333, "vocab": 50021, "dtype": "f32", "pad": 3, "top": 10,
         "masked": 0.3, "without": 9},
        # every position of a 4096-token prompt over a large vocabulary: one read of the logits decides
        {"name": "logprobs_4096", **lp, "rows": 4096, "vocab": 131072, "dtype": "bf16", "pad": 0, "top": 20,
         "masked": 0.0, "without": 1},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["quant", "linear", "logprobs"])
    if op == "quant":
        k = 32 * _log_int(rng, 1, 256)
        return {"op": op, "rows": _log_int(rng, 1, min(8192, 22000000 // k)), "k": k,
                "pad": rng.choice([0, 0, 8, 8 * rng.randint(1, 800)])}
    if op == "linear":
        k = 32 * _log_int(rng, 4, 128)
        n = _log_int(rng, 64, 131072 if k <= 2688 else 65536)
        return {"op": op, "rows": _log_int(rng, 1, max(1, min(8192, 200000000000 // (n * k)))), "k": k, "n": n,
                "out": rng.choice(["bf16", "bf16", "f32"])}
    vocab = _log_int(rng, 1000, 131072)
    rows = _log_int(rng, 1, max(1, min(4096, 250000000 // vocab)))
    return {"op": op, "rows": rows, "vocab": vocab, "dtype": rng.choice(["bf16", "f32"]),
            "pad": rng.choice([0, 0, 1, 5, 64]), "top": rng.choice([0, 1, 5, 10, 20, 32]),
            "masked": rng.choice([0.0, 0.0, 0.5]), "without": rng.choice([0, 0, rows // 5])}


# The microscaled 4-bit format: blocks of 32 along K share a scale 2^(code - 127); elements are e2m1 (sign, then the
# magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6), the even one of a byte in its low half.

def _scale_exponent(amax):
    # floor(log2 of the block's largest magnitude) less 2 (6 = 1.5 x 2^2 is the largest e2m1 value)
    return torch.where(amax > 0, torch.frexp(amax).exponent - 3, -127).clamp(min=-127)


def _round_e2m1(a):
    """|a| to the nearest e2m1 magnitude, ties to the even code, 6 past the end."""
    half = (a > 0.25).float() + (a >= 0.75).float() + (a > 1.25).float() + (a >= 1.75).float()
    return 0.5 * half + (a > 2.5).float() + (a >= 3.5).float() + 2.0 * (a > 5.0).float()


def _quantised(x):
    """The values that x's 4-bit form stands for, in f32."""
    b = x.float().reshape(x.shape[0], -1, 32)
    e = _scale_exponent(b.abs().amax(2, keepdim=True))
    return (torch.copysign(_round_e2m1(torch.ldexp(b.abs(), -e)), b) * torch.ldexp(torch.ones_like(b), e)).reshape(x.shape)


def _values(codes, scales):
    """The values of packed e2m1 codes [N, K / 2] with scale codes [N, K / 32], in f32."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    c = torch.stack([codes & 15, codes >> 4], 2).reshape(codes.shape[0], -1, 32).int()
    v = table[c & 7] * (1 - 2 * (c >> 3)).float()
    return (v * torch.exp2(scales.float() - 127.0)[:, :, None]).reshape(codes.shape[0], -1)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(1000003 * (seed + 1) + 11)

    def normal(shape, std, dtype):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).mul_(std).to(dtype)

    if case["op"] == "quant":
        m, k = case["rows"], case["k"]
        # activations: channels of different sizes, a few of them large
        size = torch.exp(1.0 * torch.randn(k + case["pad"], generator=g, device=dev))
        wide = (normal((m, k + case["pad"]), 1.0, torch.float32) * size).to(torch.bfloat16)
        return {"op": "quant", "x": wide[:, :k], "out": torch.empty((m, k), dtype=torch.bfloat16, device=dev)}
    if case["op"] == "linear":
        m, k, n = case["rows"], case["k"], case["n"]
        # normal weights of deviation 1 / sqrt(k) to 4 bits: the codes and scales that a checkpoint holds
        codes = torch.empty((n, k // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((n, k // 32), dtype=torch.uint8, device=dev)
        for i in range(0, n, 16384):
            b = normal((min(16384, n - i), k // 32, 32), k ** -0.5, torch.float32)
            e = _scale_exponent(b.abs().amax(2))
            mag = _round_e2m1(torch.ldexp(b.abs(), -e[:, :, None]))
            c = torch.where(mag < 2, 2 * mag, torch.where(mag < 4, mag + 2, mag / 2 + 4)).int() + 8 * (b < 0)
            c = c.reshape(b.shape[0], -1, 2)
            codes[i:i + 16384] = (c[:, :, 0] + 16 * c[:, :, 1]).to(torch.uint8)
            scales[i:i + 16384] = (e + 127).to(torch.uint8)
        s = {"op": "linear", "x": normal((m, k), 1.0, torch.bfloat16), "codes": codes, "scales": scales,
             "out": torch.empty((m, n), dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32, device=dev)}
        if own:
            import mamba2_ssm_mixer_gb300 as m2
            s["w"] = m2.mxfp4_pack(codes, scales)
        return s
    r, v, top = case["rows"], case["vocab"], case["top"]
    wide = normal((r, v + case["pad"]), 2.5, torch.float32)
    if case["masked"]:
        banned = torch.rand((1, v + case["pad"]), generator=g, device=dev) < case["masked"]
        banned[0, 0] = False
        wide.masked_fill_(banned, -math.inf)
    wide = wide.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
    # half of the tokens are among the likelier ones, as a prompt's are
    tokens = torch.randint(0, v, (r, 64), generator=g, device=dev)
    best = wide.gather(1, tokens).float().argmax(1)
    at = torch.where(torch.rand(r, generator=g, device=dev) < 0.5, best, 0)
    tokens = tokens.gather(1, at[:, None])[:, 0]
    if case["masked"]:
        tokens = torch.where(banned[0][tokens], 0, tokens)
    tokens[torch.randperm(r, generator=g, device=dev)[:case["without"]]] = -1
    out = {"logprobs": torch.empty(r, dtype=torch.float32, device=dev),
           "ranks": torch.empty(r, dtype=torch.int32, device=dev),
           "entropy": torch.empty(r, dtype=torch.float32, device=dev),
           "top_tokens": torch.empty((r, top), dtype=torch.int32, device=dev),
           "top_logprobs": torch.empty((r, top), dtype=torch.float32, device=dev)}
    return {"op": "logprobs", "logits": wide[:, :v], "tokens": tokens.int(), "top": top, "out": out}


def _quant_plain(s):
    s["out"].copy_(_quantised(s["x"]))
    return s["out"]


def _linear_plain(s):
    s["out"].copy_(_quantised(s["x"]) @ _values(s["codes"], s["scales"]).T)
    return s["out"]


def _logprobs_plain(s):
    x, t = s["logits"].float(), s["tokens"].long()
    v, top = x.shape[1], s["top"]
    m = x.amax(1, keepdim=True)
    d = x - m
    p = torch.exp(d)
    z = p.sum(1, dtype=torch.float64)
    logz = z.log()
    spread = (p * torch.where(p > 0, d, 0.0)).sum(1, dtype=torch.float64) / z
    col = torch.arange(v, device=x.device)
    mine = x.gather(1, t.clamp(min=0)[:, None])
    ahead = (x > mine) | ((x == mine) & (col < t[:, None]))
    out = {"logprobs": torch.where(t < 0, 0.0, (mine - m)[:, 0].double() - logz).float(),
           "ranks": torch.where(t < 0, 0, 1 + ahead.sum(1)).int(), "entropy": (logz - spread).float()}
    # the largest logits, equal ones by the lower token: whole numbers that order like (logit, -token)
    bits = (x + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, -2147483648 - bits, bits) * v + (v - 1 - col)
    token = v - 1 - torch.topk(order, top, dim=1).values % v
    out["top_tokens"] = token.int()
    out["top_logprobs"] = (d.gather(1, token).double() - logz[:, None]).float()
    return out


def run(state):
    s = state
    if own:
        import mamba2_ssm_mixer_gb300 as m2
        if s["op"] == "quant":
            return m2.mxfp4_dequant(m2.mxfp4_quant(s["x"]), out=s["out"])
        if s["op"] == "linear":
            return m2.mxfp4_linear_bf16(s["x"], s["w"], y=s["out"])
        o = m2.m2_token_logprobs(s["logits"], s["tokens"], s["top"], out=m2.TokenLogprobs(**s["out"]))
        return o._asdict()
    return {"quant": _quant_plain, "linear": _linear_plain, "logprobs": _logprobs_plain}[s["op"]](s)


def work(case):
    if case["op"] == "quant":
        return {"bytes": 4 * case["rows"] * case["k"], "flops": 4 * case["rows"] * case["k"]}
    if case["op"] == "linear":
        m, k, n = case["rows"], case["k"], case["n"]
        return {"bytes": 2 * m * k + n * k // 2 + n * k // 32 + m * n * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * m * k * n}
    read = case["rows"] * case["vocab"]
    return {"bytes": read * (2 if case["dtype"] == "bf16" else 4) + case["rows"] * (16 + 8 * case["top"]),
            "flops": 5 * read}


def _exact_blocks(x):
    """The 4-bit form's values in 64 bits, from the definition: the nearest of the fifteen values of each block."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    b = x.double().reshape(x.shape[0], -1, 32)
    amax = b.abs().amax(2, keepdim=True)
    e = ((amax.view(torch.int64) >> 52) - 1023 - 2).clamp(min=-127)     # (the exponent bits of a double)
    scale = torch.exp2(e.double())
    a = b.abs() / scale
    lo = (a[..., None] >= grid).sum(-1) - 1
    hi = (lo + 1).clamp(max=7)
    below, above = a - grid[lo], grid[hi] - a
    up = (below > above) | ((below == above) & (lo % 2 == 1))
    return (torch.where(up, grid[hi], grid[lo]) * b.sign() * scale).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quant":
        return torch.cat([_exact_blocks(rows) for rows in s["x"].split(1024)])
    if case["op"] == "linear":
        a = torch.cat([_exact_blocks(rows) for rows in s["x"].split(1024)])
        out = []
        for codes, scales in zip(s["codes"].split(8192), s["scales"].split(8192)):
            nib = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.int64, device=codes.device)
            nib[:, 0::2], nib[:, 1::2] = codes.long() % 16, codes.long() // 16
            exponent, mantissa = nib % 8 // 2, nib % 2
            mag = torch.where(exponent == 0, 0.5 * mantissa, torch.exp2(exponent.double() - 1) * (1 + 0.5 * mantissa))
            w = mag * torch.where(nib > 7, -1.0, 1.0) * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)
            out.append(a @ w.T)
        return torch.cat(out, 1)
    top, parts = case["top"], []
    step = max(1, 40000000 // case["vocab"])
    for x, t in zip(s["logits"].split(step), s["tokens"].long().split(step)):
        logp = torch.log_softmax(x.double(), 1)
        p = logp.exp()
        h = -torch.where(p > 0, p * logp, 0.0).sum(1)
        best, at = x.double().sort(dim=1, descending=True, stable=True)
        mine = logp.gather(1, t.clamp(min=0)[:, None])[:, 0]
        # the token's place in the sorted row
        place = (at == t[:, None]).int().argmax(1) + 1
        none = t < 0
        parts.append((torch.where(none, 0.0, mine), torch.where(none, 0, place).int(), h, at[:, :top].int(),
                      logp.gather(1, at[:, :top])))
    names = ("logprobs", "ranks", "entropy", "top_tokens", "top_logprobs")
    return {name: torch.cat(rows) for name, rows in zip(names, zip(*parts))}
