"""Cases of the operators that serve many requests on one mixer stack: low-rank adapters beside the shared
projections (``m2_lora_add``), beam selection over beams and vocabulary (``m2_beam_select``) and the reordering of
the paged recurrent states after it (``m2_state_reorder``).

With ``own`` false ``run`` computes them in plain torch; with ``own`` true it calls the package."""
import math

import numpy as np
import torch

own = False

# one state row of a layer: [heads, head dim, d_state], and its conv window [conv channels, width - 1]
STATE_ROW, CONV_ROW = (64, 64, 128), (6144, 3)


def listed():
    lora = {"op": "lora"}
    beam = {"op": "beam"}
    state = {"op": "state"}
    return [
        # one row of one request through in_proj with its adapter: latency alone
        {"name": "lora_decode_1", **lora, "rows": 1, "k": 2688, "n": 10304, "rank": 16, "adapters": 8, "runs": False,
         "bare": 0},
        # a decode batch in which every row has an adapter of its own (the 64-row decode workload, in_proj)
        {"name": "lora_decode_64", **lora, "rows": 64, "k": 2688, "n": 10304, "rank": 16, "adapters": 64, "runs": False,
         "bare": 0},
        # a larger decode batch sharing a few adapters of a higher rank, some rows without one (out_proj)
        {"name": "lora_decode_128_r64", **lora, "rows": 128, "k": 4096, "n": 2688, "rank": 64, "adapters": 24,
         "runs": False, "bare": 13},
        # a ragged prefill (4096 + 1024 + 512 + 37 tokens' worth of rows in runs, out_proj)
        {"name": "lora_prefill_5669_r32", **lora, "rows": 5669, "k": 4096, "n": 2688, "rank": 32, "adapters": 4,
         "runs": True, "bare": 0},
        # the 4 x 2048 prefill through in_proj, one adapter a sequence: the bytes of y decide
        {"name": "lora_prefill_8192", **lora, "rows": 8192, "k": 2688, "n": 10304, "rank": 16, "adapters": 4,
         "runs": True, "bare": 0},
        # one request, four beams: latency alone
        {"name": "beam_1x4", **beam, "batch": 1, "beams": 4, "vocab": 32000, "k": 4, "dtype": "bf16", "pad": 0,
         "done": 0, "masked": 0.0},
        # odd vocabulary in padded rows, banned tokens, finished beams
        {"name": "beam_7x5_odd", **beam, "batch": 7, "beams": 5, "vocab": 50021, "k": 10, "dtype": "f32", "pad": 3,
         "done": 4, "masked": 0.3},
        # twice as many candidates as beams, f32 logits
        {"name": "beam_16x4_f32", **beam, "batch": 16, "beams": 4, "vocab": 65536, "k": 8, "dtype": "f32", "pad": 0,
         "done": 0, "masked": 0.0},
        # a large batch over a large vocabulary: one read of the logits decides
        {"name": "beam_64x8", **beam, "batch": 64, "beams": 8, "vocab": 131072, "k": 8, "dtype": "bf16", "pad": 0,
         "done": 40, "masked": 0.0},
        # one request, four beams, one layer: two rows copied
        {"name": "state_1x4", **state, "batch": 1, "beams": 4, "layers": 1, "slots": 8, "kept": 2, "dtype": "f32"},
        # the 64-row decode workload's pool of 256 slots, half of the beams replaced
        {"name": "state_8x8", **state, "batch": 8, "beams": 8, "layers": 1, "slots": 256, "kept": 4, "dtype": "f32"},
        # all layers of the stack in one call, bf16 states
        {"name": "state_16x4_23", **state, "batch": 16, "beams": 4, "layers": 23, "slots": 64, "kept": 2,
         "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["lora", "beam", "state"])
    if op == "lora":
        rows = _log_int(rng, 1, 8192)
        return {"op": op, "rows": rows, "k": 16 * _log_int(rng, 16, 256 if rows < 4096 else 168),
                "n": _log_int(rng, 64, 10304), "rank": 8 * rng.choice([1, 2, 3, 4, 8]),
                "adapters": _log_int(rng, 1, 64), "runs": rows > 256 or rng.random() < 0.3,
                "bare": rng.choice([0, 0, rows // 7])}
    if op == "beam":
        beams = rng.randint(1, 8)
        vocab = _log_int(rng, 1000, 131072)
        k = rng.choice([beams, 2 * beams])
        batch = _log_int(rng, 1, max(1, min(64, 60000000 // (2 * beams * vocab))))
        return {"op": op, "batch": batch, "beams": beams, "vocab": vocab, "k": k, "dtype": rng.choice(["bf16", "f32"]),
                "pad": rng.choice([0, 0, 1, 5, 64]), "done": rng.choice([0, batch * beams // 5]),
                "masked": rng.choice([0.0, 0.0, 0.5])}
    batch, beams = _log_int(rng, 1, 16), rng.randint(2, 8)
    layers = _log_int(rng, 1, max(1, min(23, 1000 // (batch * beams))))
    return {"op": op, "batch": batch, "beams": beams, "layers": layers, "slots": batch * beams + rng.randint(0, 32),
            "kept": rng.randint(1, beams - 1), "dtype": rng.choice(["f32", "bf16"])}


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(1000003 * (seed + 1) + 7)
    host = np.random.default_rng(seed)

    def normal(shape, std, dtype):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).mul_(std).to(dtype)

    if case["op"] == "lora":
        m, k, n, r, na = case["rows"], case["k"], case["n"], case["rank"], case["adapters"]
        # row m names adapter ids[m]: runs of rows (the tokens of one sequence) or any order, some rows without one
        ids = np.sort(np.arange(m) % na) if case["runs"] else host.permutation(np.arange(m) % na)
        ids = host.permutation(na)[ids].astype(np.int32)
        ids[host.permutation(m)[:case["bare"]]] = -1
        return {"op": "lora", "x": normal((m, k), 1.0, torch.bfloat16), "y": normal((m, n), 1.0, torch.bfloat16),
                "a": normal((na, r, k), k ** -0.5, torch.bfloat16), "b": normal((na, n, r), r ** -0.5, torch.bfloat16),
                "scale": torch.rand(na, generator=g, device=dev) + 0.5, "ids": torch.from_numpy(ids).to(dev),
                "out": torch.empty((m, n), dtype=torch.bfloat16, device=dev)}
    if case["op"] == "beam":
        nb, kb, v = case["batch"], case["beams"], case["vocab"]
        wide = normal((nb * kb, v + case["pad"]), 2.5, torch.float32)
        if case["masked"]:
            wide.masked_fill_(torch.rand((1, v + case["pad"]), generator=g, device=dev) < case["masked"], -math.inf)
        wide = wide.to(torch.bfloat16 if case["dtype"] == "bf16" else torch.float32)
        done = np.zeros(nb * kb, bool)
        done[host.permutation(nb * kb)[:case["done"]]] = True
        return {"op": "beam", "logits": wide[:, :v], "k": case["k"], "eos": 2 if case["done"] else None,
                "scores": -4.0 * torch.rand((nb, kb), generator=g, device=dev) - 10.0,
                "done": torch.from_numpy(done.reshape(nb, kb)).to(dev) if case["done"] else None}
    nb, kb, layers = case["batch"], case["beams"], case["layers"]
    ssm = normal((layers, case["slots"], *STATE_ROW), 0.1, torch.float32 if case["dtype"] == "f32" else torch.bfloat16)
    conv = normal((layers, case["slots"], *CONV_ROW), 1.0, torch.bfloat16)
    # each request goes on with `kept` of its beams; the others' rows take further copies of those
    parents = np.empty((nb, kb), np.int32)
    for i in range(nb):
        keep = host.permutation(kb)[:case["kept"]]
        parents[i] = host.permutation(np.concatenate([keep, keep[host.integers(0, len(keep), kb - len(keep))]]))
    slots = host.permutation(case["slots"])[:nb * kb].reshape(nb, kb).astype(np.int32)
    return {"op": "state", "ssm": ssm, "conv": conv, "parents": torch.from_numpy(parents).to(dev),
            "slots": torch.from_numpy(slots).to(dev), "ssm_pools": list(ssm.unbind(0)),
            "conv_pools": list(conv.unbind(0)), "new": torch.empty_like(torch.from_numpy(slots).to(dev))}


def _lora_plain(s):
    na, r, k = s["a"].shape
    n = s["b"].shape[1]
    # x through every adapter's A; each row keeps its own adapter's part and goes through all B at once
    t = (s["x"].float() @ s["a"].float().reshape(na * r, k).T).reshape(-1, na, r)
    mine = s["ids"][:, None] == torch.arange(na, device=t.device)
    t = torch.where(mine[:, :, None], t * s["scale"][:, None], 0.0).reshape(-1, na * r)
    s["out"].copy_(s["y"].float() + t @ s["b"].float().transpose(1, 2).reshape(na * r, n))
    return s["out"]


def _beam_plain(s):
    (nb, kb), v, k = s["scores"].shape, s["logits"].shape[1], s["k"]
    x = s["logits"].float()
    x = torch.where(x.isnan(), -math.inf, x) + 0.0
    top = x.amax(1, keepdim=True)
    lse = top.double() + torch.exp(x - top).sum(1, keepdim=True, dtype=torch.float64).log()
    # the k best tokens of each beam, equal logits by the lower token: whole numbers that order like (logit, -token)
    bits = x.view(torch.int32).long()
    order = torch.where(bits < 0, -2147483648 - bits, bits) * v + torch.arange(v - 1, -1, -1, device=x.device)
    token = v - 1 - torch.topk(order, min(k, v), dim=1).values % v
    value = s["scores"].reshape(-1, 1).double() + (x.gather(1, token).double() - lse)
    if s["done"] is not None:
        # a finished beam goes on as itself: one candidate, its score unchanged
        first = torch.arange(token.shape[1], device=x.device) == 0
        ended = s["done"].reshape(-1, 1)
        value = torch.where(ended, torch.where(first, s["scores"].reshape(-1, 1).double(), -math.inf), value)
        token = torch.where(ended & first, s["eos"], token)
    flat = (token + v * torch.arange(kb, device=x.device).repeat(nb)[:, None]).reshape(nb, -1)
    flat, at = flat.sort(1)
    value, at = value.reshape(nb, -1).gather(1, at).sort(dim=1, descending=True, stable=True)
    value, flat = value[:, :k], flat.gather(1, at)[:, :k]
    none = value == -math.inf
    parents = torch.where(none, -1, flat // v)
    token = torch.where(none, -1, flat % v)
    out = {"tokens": token.int(), "parents": parents.int(), "scores": value.float()}
    if s["done"] is not None:
        out["done"] = (s["done"].gather(1, parents.clamp(min=0)) & ~none) | (token == s["eos"])
    return out


def _state_plain(s):
    slots, parents = s["slots"].long(), s["parents"].long()
    beam = torch.arange(slots.shape[1], device=slots.device)
    same = parents[:, :, None] == parents[:, None, :]
    first = ~(same & (beam[None, :] < beam[:, None])).any(2)
    # the first child of a beam keeps its slot; the others take, in order, the slots of beams that have no child
    childless = ~(parents[:, :, None] == beam).any(1)
    wanted = torch.where(first, -1, (~first).long().cumsum(1) - 1)
    offered = torch.where(childless, childless.long().cumsum(1) - 1, -2)
    given = ((wanted[:, :, None] == offered[:, None, :]).long() * slots[:, None, :]).sum(2)
    old = slots.gather(1, parents)
    new = torch.where(first, old, given)
    s["ssm"][:, new.reshape(-1)] = s["ssm"][:, old.reshape(-1)]
    s["conv"][:, new.reshape(-1)] = s["conv"][:, old.reshape(-1)]
    s["new"].copy_(new)
    return {"slots": s["new"], "ssm": s["ssm"], "conv": s["conv"]}


def run(state):
    s = state
    if own:
        import mamba2_ssm_mixer_gb300 as m2
        if s["op"] == "lora":
            return m2.m2_lora_add(s["y"], s["x"], s["a"], s["b"], s["ids"], scale=s["scale"], out=s["out"])
        if s["op"] == "beam":
            step = m2.m2_beam_select(s["logits"], s["scores"], s["k"], eos_token=s["eos"], done=s["done"])
            out = {"tokens": step.tokens, "parents": step.parents, "scores": step.scores}
            return out if s["done"] is None else {**out, "done": step.done}
        m2.m2_state_reorder(s["conv_pools"], s["ssm_pools"], s["slots"], s["parents"], out=s["new"])
        return {"slots": s["new"], "ssm": s["ssm"], "conv": s["conv"]}
    return {"lora": _lora_plain, "beam": _beam_plain, "state": _state_plain}[s["op"]](s)


def work(case):
    if case["op"] == "lora":
        m, k, n, r = case["rows"], case["k"], case["n"], case["rank"]
        named = min(case["adapters"], m)
        return {"bytes": 2 * (m - case["bare"]) * k + 4 * m * n + 2 * named * r * (k + n) + 4 * m + 4 * named,
                "flops": 2 * (m - case["bare"]) * r * (k + n)}
    if case["op"] == "beam":
        rows = case["batch"] * case["beams"]
        read = (rows - case["done"]) * case["vocab"]
        return {"bytes": read * (2 if case["dtype"] == "bf16" else 4) + 5 * rows + 13 * case["batch"] * case["k"],
                "flops": 3 * read}
    row = math.prod(STATE_ROW) * (4 if case["dtype"] == "f32" else 2) + math.prod(CONV_ROW) * 2
    copies = case["batch"] * (case["beams"] - case["kept"]) * case["layers"]
    return {"bytes": 2 * copies * row + 12 * case["batch"] * case["beams"], "flops": 0}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lora":
        out = s["y"].double()
        for i in range(case["adapters"]):
            at = torch.nonzero(s["ids"] == i).reshape(-1)
            down = s["x"][at].double() @ s["a"][i].double().T
            out[at] += s["scale"][i].double() * (down @ s["b"][i].double().T)
        return out
    if case["op"] == "beam":
        (nb, kb), v, k = s["scores"].shape, case["vocab"], case["k"]
        got = {"tokens": [], "parents": [], "scores": [], "done": []}
        for i in range(nb):
            x = s["logits"][i * kb:(i + 1) * kb].double()
            value = s["scores"][i].double()[:, None] + torch.log_softmax(x, 1)
            if s["done"] is not None:
                for j in torch.nonzero(s["done"][i]).reshape(-1).tolist():
                    value[j] = -math.inf
                    value[j, s["eos"]] = s["scores"][i, j].double()
            best, at = value.reshape(-1).sort(descending=True, stable=True)
            best, at = best[:k], at[:k]
            dead = best == -math.inf
            token, parent = torch.where(dead, -1, at % v), torch.where(dead, -1, at // v)
            got["tokens"].append(token.int())
            got["parents"].append(parent.int())
            got["scores"].append(best)
            if s["done"] is not None:
                got["done"].append((token == s["eos"]) | (s["done"][i][parent.clamp(min=0)] & ~dead))
        return {name: torch.stack(rows) for name, rows in got.items() if rows}
    slots, parents = s["slots"].tolist(), s["parents"].tolist()
    new, moves = [], []
    for row, par in zip(slots, parents):
        spare = [row[j] for j in range(len(row)) if j not in par]
        seen = set()
        now = []
        for p in par:
            if p not in seen:
                now.append(row[p])
            else:
                now.append(spare.pop(0))
                moves.append((now[-1], row[p]))
            seen.add(p)
        new.append(now)
    for to, of in moves:
        s["ssm"][:, to] = s["ssm"][:, of]
        s["conv"][:, to] = s["conv"][:, of]
    return {"slots": torch.tensor(new, dtype=torch.int32, device=s["ssm"].device), "ssm": s["ssm"], "conv": s["conv"]}
