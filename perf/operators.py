"""The serving operators' measured cases: the expert layer of a few tokens
(moe_ffn_decode) and low-rank adapters beside a shared projection
(lora_linear), each with its plain form in elementary torch operations and its
definition in 64 bits.
"""
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
CODE = {"f32": 0, "f16": 1, "bf16": 2}
NO_ADAPTER = 0xFFFFFFFF


def listed():
    return [
        # one generated token through a layer of 128 small experts: the decode step of one user
        moe("moe one token", "bf16", 1, 2048, 768, 8, 128),
        # the same step in a large model: 256 experts of 1536 x 4096 (the decode benchmark's experts)
        moe("moe one token, large", "bf16", 1, 4096, 1536, 8, 256),
        # the smallest layer (draft models, tests): latency alone
        moe("moe small layer", "f16", 1, 256, 96, 4, 16),
        # eight users decoding together: about 50 of 128 experts, most with one or two rows
        moe("moe 8 tokens", "f16", 8, 2048, 768, 8, 128),
        # a full decode batch: nearly every expert, with popular experts as trained routers have them
        moe("moe 64 tokens, skewed", "bf16", 64, 2048, 768, 8, 128, skew=0.5),
        # sizes off every tile, 32-bit weights, gates not renormalised, no selection bias
        moe("moe odd sizes", "f32", 13, 1001, 363, 5, 37, bias=False, renorm=False),
        # one user's token through a square projection with that user's adapter
        lora("lora one token", "bf16", "bf16", 1, 4096, 4096, 16, 64),
        # a decode batch of 32 users, nearly all with adapters of their own and of mixed ranks
        lora("lora 32 tokens, mixed", "bf16", "bf16", 32, 1536, 4096, 64, 128, mixed=True, none=0.1),
        # sizes off every tile, 32-bit adapters beside f16 weights, a third of the rows without one
        lora("lora odd sizes", "f16", "f32", 9, 1111, 1003, 11, 8, mixed=True, none=0.33),
        # a prompt chunk of four requests in the fixed f32 order
        lora("lora chunk", "bf16", "bf16", 512, 768, 2048, 16, 8, requests=4),
        # prompts of eight requests in the split-16 arithmetic: the largest projection
        lora("lora prompts", "bf16", "bf16", 2048, 4096, 4096, 32, 16, requests=8, arith="split16"),
        # adapters added to rows that another product (the experts' down projection) has made
        lora("lora on given rows", "f16", "f16", 16384, 2048, 768, 16, 32, requests=48, none=0.1, given=True),
    ]


def moe(name, dtype, m, hidden, inter, top_k, experts, bias=True, renorm=True, skew=0.0):
    return {"name": name, "op": "moe", "dtype": dtype, "m": m, "hidden": hidden, "inter": inter, "top_k": top_k,
            "experts": experts, "bias": bias, "renorm": renorm, "skew": skew}


def lora(name, dtype, adapter_dtype, m, n, k, rank, adapters, mixed=False, none=0.0, requests=0, arith="f32",
         given=False):
    """requests: the rows are that many runs of consecutive rows (prompts), 0: every row is a request of its own."""
    return {"name": name, "op": "lora", "dtype": dtype, "adapter_dtype": adapter_dtype, "m": m, "n": n, "k": k,
            "rank": rank, "adapters": adapters, "mixed": mixed, "none": none, "requests": requests, "arith": arith,
            "given": given}


def draw(rng):
    def spread(lo, hi):
        return min(hi, max(lo, round(lo * (hi / lo) ** rng.random())))

    def size(lo, hi, step):
        """A length, a multiple of `step` in half of the draws and any number in the others."""
        v = spread(lo, hi)
        return max(step, v // step * step) if rng.random() < 0.5 else v

    if rng.random() < 0.5:
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        experts = spread(4, 256)
        hidden, inter = size(128, 4096, 64), size(64, 1536, 32)
        top_k = min(rng.choice([1, 2, 4, 6, 8, 8]), experts)
        m = spread(1, 64)
        case = moe(None, dtype, m, hidden, inter, top_k, experts, bias=rng.random() < 0.7,
                   renorm=rng.random() < 0.8, skew=rng.choice([0.0, 0.5, 1.5]))
    else:
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        arith = "split16" if dtype != "f32" and rng.random() < 0.4 else "f32"
        given = rng.random() < 0.25
        k, n = size(64, 4096, 64), size(64, 4096, 64)
        if arith == "split16":
            k = k // 8 * 8
        m = spread(1, 8192) if given else spread(1, 2048)
        case = lora(None, dtype, rng.choice([dtype, dtype, "f32"]), m, n, k, spread(1, 64), spread(1, 128),
                    mixed=rng.random() < 0.5, none=rng.choice([0.0, 0.1, 0.5]),
                    requests=0 if m < 64 else spread(1, 64), arith=arith, given=given)
    del case["name"]
    most = max(cost(c) for c in listed())
    while cost(case) > most and case["m"] > 1:
        case["m"] = case["m"] // 2
    return case


def cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def work(case):
    """Distinct experts and adapters are counted as expected: a token takes top_k of the experts, a request one adapter."""
    c, m = case, case["m"]
    if c["op"] == "moe":
        e, rows = c["experts"], m * c["top_k"]
        touched = e * (1 - (1 - c["top_k"] / e) ** m)
        weight = 3 * c["hidden"] * c["inter"]
        return {"bytes": touched * weight * SIZE[c["dtype"]] + 8 * m * c["hidden"] + 4 * m * e + 8 * rows,
                "flops": 2 * rows * weight}
    requests = c["requests"] or m
    used = c["adapters"] * (1 - (1 - 1 / c["adapters"]) ** (requests * (1 - c["none"])))
    rank = c["rank"] * (0.5 if c["mixed"] else 1.0)
    rows = m * (1 - c["none"])
    base = 4 * m * c["n"] if c["given"] else c["n"] * c["k"] * SIZE[c["dtype"]]
    flops = 2 * rows * rank * (c["n"] + c["k"]) + (0 if c["given"] else 2 * m * c["n"] * c["k"])
    return {"bytes": base + 4 * m * (c["n"] + c["k"]) + used * rank * (c["n"] + c["k"]) * SIZE[c["adapter_dtype"]],
            "flops": flops}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c, dev = case, "cuda"

    def normal(std, *shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype).mul_(std)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device=dev)

    s = {"case": c}
    if c["op"] == "moe":
        dt, e, h, i, m = DTYPES[c["dtype"]], c["experts"], c["hidden"], c["inter"], c["m"]
        s["w_gate"] = normal(h ** -0.5, e, i, h, dtype=dt)
        s["w_up"] = normal(h ** -0.5, e, i, h, dtype=dt)
        s["w_down"] = normal(i ** -0.5, e, h, i, dtype=dt)
        s["x"] = normal(1.0, m, h)
        s["logits"] = normal(1.0, m, e) + c["skew"] * normal(1.0, e)
        s["bias"] = uniform(e) * 0.2 - 0.1 if c["bias"] else None
        s["ids"] = torch.zeros(m, c["top_k"], dtype=torch.int32, device=dev)
        s["gates"] = torch.zeros(m, c["top_k"], device=dev)
        s["out"] = torch.zeros(m, h, device=dev)
        if own:
            from expert_id_matmul_amd import binding as B
            s["lib"] = B.load()
            s["shape"] = B.make_ffn_shape(CODE[c["dtype"]], m, h, i, c["top_k"], e)
            s["scratch"] = torch.empty(s["lib"].moe_ffn_decode_scratch_bytes(s["shape"]), dtype=torch.uint8, device=dev)
        return s
    dt, da, m, n, k, r, a = (DTYPES[c["dtype"]], DTYPES[c["adapter_dtype"]], c["m"], c["n"], c["k"], c["rank"],
                             c["adapters"])
    s["x"] = normal(1.0, m, k)
    s["w"] = None if c["given"] else normal(k ** -0.5, n, k, dtype=dt)
    s["base"] = normal(1.0, m, n) if c["given"] else None
    s["a"] = normal(k ** -0.5, a, r, k, dtype=da)
    s["b"] = normal(r ** -0.5, a, n, r, dtype=da)
    s["ranks"] = (1 + (uniform(a) * r).int()).clamp(max=r) if c["mixed"] else None
    s["scales"] = 0.25 + uniform(a)
    requests = c["requests"] or m
    ids = (uniform(requests) * a).int().clamp(max=a - 1)
    ids = torch.where(uniform(requests) < c["none"], torch.full_like(ids, -1), ids)  # -1: NO_ADAPTER's bits
    if c["requests"]:  # prompts of uneven lengths
        cuts = (uniform(requests - 1) * m).int().sort().values
        ids = ids[torch.searchsorted(cuts, torch.arange(m, device=dev, dtype=torch.int32), right=True)]
    s["ids"] = ids.contiguous()
    s["y"] = torch.zeros(m, n, device=dev)
    if own:
        from expert_id_matmul_amd import binding as B
        s["lib"] = B.load()
        s["shape"] = B.make_lora_shape(CODE[c["dtype"]], CODE[c["adapter_dtype"]], m, n, k, a, r,
                                       arith=B.ARITH_SPLIT16 if c["arith"] == "split16" else B.ARITH_F32)
        s["scratch"] = torch.empty(s["lib"].lora_linear_scratch_bytes(s["shape"]), dtype=torch.uint8, device=dev)
    return s


def run(state):
    return run_moe(state) if state["case"]["op"] == "moe" else run_lora(state)


def run_moe(s):
    c = s["case"]
    if own:
        s["lib"].moe_ffn_decode(s["shape"], s["w_gate"], s["w_up"], s["w_down"], s["x"], s["logits"], s["bias"],
                                s["ids"], s["gates"], s["out"], s["scratch"], renormalize=c["renorm"])
        return {"ids": s["ids"], "gates": s["gates"], "out": s["out"]}
    score = torch.sigmoid(s["logits"].double()).float()
    key = score if s["bias"] is None else score + s["bias"]
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, : c["top_k"]]
    gates = torch.gather(score, 1, ids)
    if c["renorm"]:
        gates = gates / gates.sum(1, keepdim=True)
    flat = ids.reshape(-1)
    x = s["x"].repeat_interleave(c["top_k"], 0).unsqueeze(2)
    gate = torch.bmm(s["w_gate"][flat].float(), x)
    up = torch.bmm(s["w_up"][flat].float(), x)
    h = gate / (1 + torch.exp(-gate)) * up
    y = torch.bmm(s["w_down"][flat].float(), h).view(c["m"], c["top_k"], c["hidden"])
    return {"ids": ids.int(), "gates": gates, "out": (gates.unsqueeze(2) * y).sum(1)}


def run_lora(s):
    c = s["case"]
    if own:
        s["lib"].lora_linear(s["shape"], s["w"], s["base"], s["a"], s["b"], s["ranks"], s["scales"], s["x"], s["ids"],
                             s["y"], s["scratch"])
        return s["y"]
    y = s["base"] if c["given"] else s["x"] @ s["w"].float().t()
    has = s["ids"] >= 0
    at = s["ids"].clamp(min=0).long()
    v = torch.bmm(s["a"][at].float(), s["x"].unsqueeze(2))
    if s["ranks"] is not None:
        live = torch.arange(c["rank"], device=v.device) < s["ranks"][at].unsqueeze(1)
        v = v * live.unsqueeze(2)
    u = torch.bmm(s["b"][at].float(), v).squeeze(2)
    return y + torch.where(has, s["scales"][at], torch.zeros_like(s["scales"][at])).unsqueeze(1) * u


def exact(case, seed):
    """The operators' definitions in 64 bits, expert by expert and adapter by adapter."""
    s, c = prepare(case, seed), case
    x = s["x"].double()
    if c["op"] == "moe":
        # the scores are 32-bit numbers by definition: the selection compares those
        p = (1 / (1 + torch.exp(-s["logits"].double()))).float()
        key = p + s["bias"] if s["bias"] is not None else p
        left, picks = key.clone(), []
        for _ in range(c["top_k"]):
            picks.append(torch.argmax((left == left.max(1, keepdim=True).values).int(), 1))
            left[torch.arange(c["m"], device=x.device), picks[-1]] = -float("inf")
        ids = torch.stack(picks, 1)
        gates = torch.gather(p, 1, ids).double()
        if c["renorm"]:
            gates = gates / gates.sum(1, keepdim=True)
        out = torch.zeros(c["m"], c["hidden"], dtype=torch.float64, device=x.device)
        for e in ids.unique().tolist():
            t, slot = (ids == e).nonzero(as_tuple=True)
            gate = x[t] @ s["w_gate"][e].double().t()
            h = gate * torch.sigmoid(gate) * (x[t] @ s["w_up"][e].double().t())
            out.index_add_(0, t, gates[t, slot].unsqueeze(1) * (h @ s["w_down"][e].double().t()))
        return {"ids": None, "gates": gates, "out": out}
    y = s["base"].double().clone() if c["given"] else x @ s["w"].double().t()
    for a in s["ids"].unique().tolist():
        if a < 0:
            continue
        t = (s["ids"] == a).nonzero(as_tuple=True)[0]
        r = c["rank"] if s["ranks"] is None else int(s["ranks"][a])
        low = x[t] @ s["a"][a, :r].double().t()
        y[t] += s["scales"][a].double() * (low @ s["b"][a, :, :r].double().t())
    return y
