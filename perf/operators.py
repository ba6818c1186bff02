"""Cases for the operators of quantised decoding: the expert router, the mixture-of-experts layer on packed weights,
and the log probabilities behind an LM head.

``listed()`` and ``draw()`` give cases, ``prepare()`` what a program holds before the call, ``run()`` one pass: the
operators in plain torch where ``own`` is false, the framework's calls where it is true.  ``exact()`` is the same
result in 64 bits, written apart from the plain form."""
import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"fp16": 2, "bf16": 2, "fp32": 4}


def _moe(name, T, E, k, K, I, N, bits, G, dtype, frac=False, act="silu", empty=False):
    return {"name": name, "op": "moe", "T": T, "E": E, "k": k, "K": K, "I": I, "N": N, "bits": bits, "G": G,
            "dtype": dtype, "frac": frac, "act": act, "empty": empty}


def _route(name, T, E, k, dtype, renormalize=True):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "dtype": dtype, "renormalize": renormalize}


def _logprobs(name, R, V, top, dtype, masked=0.0):
    return {"name": name, "op": "logprobs", "R": R, "V": V, "top": top, "dtype": dtype, "masked": masked}


def listed():
    return [
        # one sequence being decoded through a layer of many small experts: launch and latency bound
        _moe("moe 1 token, 8 of 64", 1, 64, 8, 2048, 1024, 2048, 4, 128, "fp16"),
        # a batch of sequences decoded through a few large experts: every expert is read
        _moe("moe 16 tokens, 2 of 8", 16, 8, 2, 4096, 11008, 4096, 4, 128, "bf16"),
        # a wide batch over many experts, a few tokens on each, 8-bit words, fractional zero points
        _moe("moe 48 tokens, 8-bit", 48, 32, 4, 2048, 1408, 2048, 8, 128, "fp16", frac=True),
        # a small ragged layer: odd token count, per-channel scales, a K that ends inside a tile, some empty slots
        _moe("moe ragged", 5, 12, 3, 1112, 744, 1000, 4, -1, "bf16", act="gelu", empty=True),
        # the router of one decoded token, and of a prompt
        _route("route 1 token", 1, 64, 8, "fp32"),
        _route("route prompt", 8192, 128, 8, "bf16"),
        _route("route many experts", 1000, 500, 10, "fp16", renormalize=False),
        # one sampled token with its five alternatives
        _logprobs("logprobs 1 row", 1, 32000, 5, "fp16"),
        # a decoded batch, a vocabulary whose rows are not 16-byte aligned
        _logprobs("logprobs 64 odd rows", 64, 50001, 20, "bf16"),
        # constrained decoding: most of the vocabulary masked out
        _logprobs("logprobs 32 masked rows", 32, 128000, 8, "fp32", masked=0.9),
        # scoring a prompt: every position of a long text
        _logprobs("logprobs prompt", 2048, 128000, 1, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["moe", "moe", "moe", "route", "logprobs", "logprobs"])
    if op == "moe":
        while True:
            bits = rng.choice([4, 4, 8])
            G = rng.choice([32, 64, 128, 128, -1])
            q = G if G > 0 else 8
            T, E = _log_int(rng, 1, 64), _log_int(rng, 2, 128)
            k = rng.randint(1, min(E, 8))
            K = max(q, _log_int(rng, 256, 8192) // q * q)
            inner = max(q, _log_int(rng, 128, 16384) // q * q)
            N = max(8, _log_int(rng, 256, 8192) // 8 * 8)
            if E * (2 * K * inner + inner * N) * bits <= 8 * 540e6:
                break
        c = _moe("", T, E, k, K, inner, N, bits, G, rng.choice(["fp16", "bf16"]), rng.random() < 0.3,
                 rng.choice(["silu", "silu", "gelu"]), rng.random() < 0.2)
    elif op == "route":
        E = _log_int(rng, 4, 512)
        c = _route("", _log_int(rng, 1, 8192), E, rng.randint(1, min(E, 16)), rng.choice(["fp16", "bf16", "fp32"]),
                   rng.random() < 0.7)
    else:
        while True:
            R, V = _log_int(rng, 1, 4096), _log_int(rng, 1000, 200000)
            dtype = rng.choice(["fp16", "bf16", "fp32"])
            if R * V * SIZE[dtype] <= 520e6:
                break
        c = _logprobs("", R, V, rng.choice([0, 1, 5, 8, 20, 32]), dtype, rng.choice([0.0, 0.0, 0.5, 0.9]))
    del c["name"]
    return c


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _packed(g, E, K, N, bits, G, dtype, frac):
    """E packed weights (K-major words), scales and zero points: the products of unit inputs have unit size."""
    eps, groups = 32 // bits, 1 if G == -1 else K // G
    w = torch.randint(-2**31, 2**31, (E, K // eps, N), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    top = 2**bits - 1
    s = (0.5 + torch.rand((E, groups, N), generator=g, device="cuda")) / (0.29 * top * math.sqrt(K))
    z = (top + 1) / 2 + torch.randn((E, groups, N), generator=g, device="cuda") * top / 16
    return w, s.to(dtype), (z if frac else z.round()).to(dtype)


def prepare(case, seed):
    g, c = _gen(seed), dict(case)
    dtype = DTYPES[c["dtype"]]
    if c["op"] == "moe":
        x = torch.randn((c["T"], c["K"]), generator=g, device="cuda").to(dtype)
        score = torch.randn((c["T"], c["E"]), generator=g, device="cuda")
        top, ids = torch.topk(score, c["k"], dim=1)
        weights, ids = torch.softmax(top, 1), ids.to(torch.int32)
        if c["empty"]:  # padded rows of a batch, and tokens routed to fewer experts
            ids[-1] = -1
            ids[0, -1] = -1
        up = _packed(g, c["E"], c["K"], 2 * c["I"], c["bits"], c["G"], dtype, c["frac"])
        down = _packed(g, c["E"], c["I"], c["N"], c["bits"], c["G"], dtype, c["frac"])
        c.update(x=x, ids=ids, weights=weights, up=up, down=down)
        if own:  # the layer that a program builds once, when it loads its weights
            import gemm_wq_gemv_b200 as wq
            c["layer"] = wq.MoePlan(*up, *down, c["bits"], c["G"], c["T"], c["k"], activation=c["act"])
    elif c["op"] == "route":
        c["logits"] = (1.5 * torch.randn((c["T"], c["E"]), generator=g, device="cuda")).to(dtype)
    else:
        R, V = c["R"], c["V"]
        logits = 2.5 * torch.randn((R, V), generator=g, device="cuda")
        likely = torch.randint(0, V, (R, 8), generator=g, device="cuda")
        logits.scatter_add_(1, likely, 5 + 7 * torch.rand((R, 8), generator=g, device="cuda"))
        if c["masked"]:
            gone = torch.rand((R, V), generator=g, device="cuda") < c["masked"]
            gone.scatter_(1, likely, False)
            logits.masked_fill_(gone, -math.inf)
            del gone
        pick = torch.randint(0, 8, (R, 1), generator=g, device="cuda")
        c["logits"], c["tokens"] = logits.to(dtype), likely.gather(1, pick)[:, 0].contiguous()
    return c


# ------------------------------------------------------------------ plain forms

def _dequant(w, s, z, bits):
    """(.., K, N) fp32 weights of packed words (.., K / eps, N)."""
    eps = 32 // bits
    shifts = torch.arange(0, 32, bits, device=w.device, dtype=torch.int32)[:, None]
    q = ((w.unsqueeze(-2) >> shifts) & (2**bits - 1)).flatten(-3, -2).float()
    G = w.shape[-2] * eps // s.shape[-2]
    q = q.unflatten(-2, (-1, G))
    return ((q - z.float().unsqueeze(-2)) * s.float().unsqueeze(-2)).flatten(-3, -2)


def _activate(g, act):
    return g / (1 + torch.exp(-g)) if act == "silu" else 0.5 * g * (1 + torch.erf(g * math.sqrt(0.5)))


def _plain_moe(c):
    T, E, k, inner = c["T"], c["E"], c["k"], c["I"]
    x, ids, used = c["x"].float(), c["ids"].long().clamp(min=0), (c["ids"] >= 0).float()
    weights = c["weights"] * used
    if T * k < E:  # fewer slots than experts: the chosen experts alone
        pick = ids.flatten()
        xs = x.repeat_interleave(k, 0)[:, None]
        gu = xs @ _dequant(*(t[pick] for t in c["up"]), c["bits"])
        h = _activate(gu[..., :inner], c["act"]) * gu[..., inner:]
        y = (h @ _dequant(*(t[pick] for t in c["down"]), c["bits"])).view(T, k, -1)
        return (y * weights[:, :, None]).sum(1).to(c["x"].dtype)
    gu = x @ _dequant(*c["up"], c["bits"])  # (E, T, 2 I)
    h = _activate(gu[..., :inner], c["act"]) * gu[..., inner:]
    y = h @ _dequant(*c["down"], c["bits"])
    mix = torch.zeros((T, E), device=x.device).scatter_add_(1, ids, weights)
    return (y * mix.t()[:, :, None]).sum(0).to(c["x"].dtype)


def _ordered(values):
    """int64 keys in the order (value descending, index ascending), for the largest of a row."""
    bits = (values + 0.0).view(torch.int32).long()
    up = torch.where(bits < 0, -(bits & 0x7FFFFFFF) - 1, bits)
    return (up << 32) - torch.arange(values.shape[1], device=values.device)


def _plain_route(c):
    l = c["logits"].float()
    ids = torch.topk(_ordered(l), c["k"], dim=1)[1]
    top = l.gather(1, ids)
    m = top[:, :1]
    e = torch.exp(top - m)
    total = e.sum(1, keepdim=True) if c["renormalize"] else torch.exp(l - m).sum(1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": e / total}


def _plain_logprobs(c):
    l = c["logits"].float()
    m = l.amax(1, keepdim=True)
    d = l - m
    e = torch.exp(d)
    total = e.sum(1)
    log_total = total.log()
    entropy = log_total - torch.where(e > 0, e * d, 0.0).sum(1) / total
    del e, d
    lse = m[:, 0] + log_total
    out = {"logprob": l.gather(1, c["tokens"][:, None])[:, 0] - lse, "entropy": entropy}
    if c["top"]:
        out["top_id"] = torch.topk(_ordered(l), c["top"], dim=1)[1]
        out["top_logprob"] = l.gather(1, out["top_id"]) - lse[:, None]
    return out


def run(state):
    c = state
    if own:
        import gemm_wq_gemv_b200 as wq
        if c["op"] == "moe":
            return c["layer"](c["x"], c["ids"], c["weights"])
        if c["op"] == "route":
            ids, weights = wq.moe_route(c["logits"], c["k"], renormalize=c["renormalize"])
            return {"ids": ids, "weights": weights}
        return wq.logprobs(c["logits"], c["tokens"], top_k=c["top"])
    return {"moe": _plain_moe, "route": _plain_route, "logprobs": _plain_logprobs}[c["op"]](c)


# ------------------------------------------------------------------ work and the 64-bit result

def work(case):
    c = case
    if c["op"] == "moe":
        T, E, k, K, inner, N, bits = (c[n] for n in ("T", "E", "k", "K", "I", "N", "bits"))
        active = E * (1 - (1 - k / E) ** T)  # experts that T tokens choose, on average: each is read once
        groups = (1 if c["G"] == -1 else K // c["G"]) * 2 * inner + (1 if c["G"] == -1 else inner // c["G"]) * N
        expert = (2 * K * inner + inner * N) * bits // 8 + 4 * groups
        return {"bytes": active * expert + 2 * T * (K + N) + 8 * T * k, "flops": 2 * T * k * (2 * K * inner + inner * N)}
    if c["op"] == "route":
        return {"bytes": c["T"] * (c["E"] * SIZE[c["dtype"]] + 8 * c["k"]), "flops": 4 * c["T"] * c["E"]}
    R, V = c["R"], c["V"]
    return {"bytes": R * (V * SIZE[c["dtype"]] + 16 + 12 * c["top"]), "flops": 6 * R * V}


def _exact_weight(w, s, z, bits, G):
    words = w.long() & 0xFFFFFFFF
    base = 2**bits
    codes = torch.stack([torch.div(words, base**j, rounding_mode="floor") % base for j in range(32 // bits)], 1)
    codes = codes.reshape(-1, w.shape[1]).double()
    K = codes.shape[0]
    group = torch.arange(K, device=w.device) // (K if G == -1 else G)
    codes -= z.double()[group]
    codes *= s.double()[group]
    return codes


def exact(case, seed):
    c = prepare(case, seed)
    if c["op"] == "moe":
        x, inner = c["x"].double(), c["I"]
        y = torch.zeros((c["T"], c["N"]), dtype=torch.float64, device="cuda")
        for e in range(c["E"]):
            token, slot = torch.nonzero(c["ids"] == e, as_tuple=True)
            if not len(token):
                continue
            gu = x[token] @ _exact_weight(*(t[e] for t in c["up"]), c["bits"], c["G"])
            gate = gu[:, :inner]
            if c["act"] == "silu":
                gate = gate * torch.sigmoid(gate)
            else:
                gate = gate * 0.5 * torch.special.erfc(-gate / math.sqrt(2.0))
            part = (gate * gu[:, inner:]) @ _exact_weight(*(t[e] for t in c["down"]), c["bits"], c["G"])
            y.index_add_(0, token, part * c["weights"][token, slot].double()[:, None])
        return y
    l = c["logits"].double()
    if c["op"] == "route":
        ids = torch.sort(l, dim=1, descending=True, stable=True)[1][:, :c["k"]]
        p = torch.softmax(l, 1).gather(1, ids)
        return {"ids": ids.to(torch.int32), "weights": p / p.sum(1, keepdim=True) if c["renormalize"] else p}
    out = {"logprob": [], "entropy": [], "top_id": [], "top_logprob": []}
    for rows, tokens in zip(l.split(256), c["tokens"].split(256)):
        logp = torch.log_softmax(rows, 1)
        out["logprob"].append(logp.gather(1, tokens[:, None])[:, 0])
        out["entropy"].append(torch.special.entr(logp.exp()).sum(1))
        if c["top"]:
            out["top_id"].append(torch.sort(rows, dim=1, descending=True, stable=True)[1][:, :c["top"]].clone())
            out["top_logprob"].append(logp.gather(1, out["top_id"][-1]))
    return {k: torch.cat(v) for k, v in out.items() if v}
