"""Cases of the operators on 8-bit activations, for timing and comparison.

Four operators, each in a plain form (elementary torch operations in 32
bits) and as the calls of the library's binding:

  tokens   fp16 or fp32 activations to int8 codes, one scale per token
  swiglu   silu(gate) * up of a gated MLP's first product, to int8 codes
  linear   int8 activations times an int8 weight, scales per token and channel
  grouped  the same with the tokens sorted by expert, one weight per expert

``own`` selects which of the two ``run`` takes.
"""
import math

import torch

own = False


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token of a ChatGLM2-6B-shaped block before its next product: the smallest call, latency alone
        {"name": "tokens decode", "op": "tokens", "M": 1, "K": 4096, "dtype": "float16"},
        # a padded prompt of 2048 tokens at the same width
        {"name": "tokens prefill", "op": "tokens", "M": 2048, "K": 4096, "dtype": "float16"},
        # activations that a host framework keeps in fp32, in a width that is no multiple of 16
        {"name": "tokens fp32 ragged", "op": "tokens", "M": 777, "K": 1000, "dtype": "float32"},
        # the gated MLP between its two products: 16 sequences decoding, and a prompt
        {"name": "swiglu decode", "op": "swiglu", "M": 16, "K": 13696},
        {"name": "swiglu prefill", "op": "swiglu", "M": 2048, "K": 13696},
        # the ChatGLM2-6B h-to-4h weight, one token
        {"name": "linear decode", "op": "linear", "M": 1, "K": 4096, "N": 27392, "asym": False, "bias": False},
        # the 4h-to-h weight with zero points, 48 sequences decoding together
        {"name": "linear batch asym", "op": "linear", "M": 48, "K": 13696, "N": 4096, "asym": True, "bias": True},
        # the h-to-4h weight over a prompt of 2048 tokens: the largest call
        {"name": "linear prefill", "op": "linear", "M": 2048, "K": 4096, "N": 27392, "asym": False, "bias": False},
        # BERT-base QKV, 4096 tokens: short sums, wide output
        {"name": "linear bert qkv", "op": "linear", "M": 4096, "K": 768, "N": 2304, "asym": False, "bias": True},
        # 8 experts of the h-to-h shape, 8 sequences decoding with two experts each
        {"name": "grouped decode", "op": "grouped", "T": 16, "behind": 0, "E": 8, "K": 4096, "N": 4096, "asym": False,
         "bias": False, "skew": 0.0},
        # odd sizes, uneven groups, some of them empty, rows behind the last group
        {"name": "grouped ragged asym", "op": "grouped", "T": 3001, "behind": 77, "E": 16, "K": 1000, "N": 1032, "asym": True,
         "bias": True, "skew": 1.5},
        # 8 experts over a prompt of 2048 tokens with two experts each
        {"name": "grouped prefill", "op": "grouped", "T": 4096, "behind": 0, "E": 8, "K": 4096, "N": 13696, "asym": False,
         "bias": False, "skew": 0.5},
    ]


def _log(rng, lo, hi, step=1):
    """A size between lo and hi, spread over its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["tokens", "swiglu", "linear", "linear", "grouped", "grouped"])
    most = max((work(c)["flops"] + 100 * work(c)["bytes"]) for c in listed() if c["op"] == op)
    while True:
        if op == "tokens":
            c = {"op": op, "M": _log(rng, 1, 4096), "K": _log(rng, 64, 16384, 8),
                 "dtype": rng.choice(["float16", "float32"])}
        elif op == "swiglu":
            c = {"op": op, "M": _log(rng, 1, 4096), "K": _log(rng, 64, 16384, 8)}
        elif op == "linear":
            c = {"op": op, "M": _log(rng, 1, 4096), "K": _log(rng, 256, 16384, 8), "N": _log(rng, 256, 27392, 8),
                 "asym": rng.random() < 0.3, "bias": rng.random() < 0.5}
        else:
            T = _log(rng, 4, 4096)
            c = {"op": op, "T": T, "behind": rng.choice([0, T // 7]), "E": _log(rng, 2, 64), "K": _log(rng, 256, 8192, 8),
                 "N": _log(rng, 256, 13696, 8), "asym": rng.random() < 0.3, "bias": rng.random() < 0.5,
                 "skew": round(rng.uniform(0.0, 1.5), 2)}
        w = work(c)
        if w["flops"] + 100 * w["bytes"] <= most:
            return c


def work(case):
    """Each input read once, each output written once; 2 operations a product."""
    if case["op"] == "tokens":
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": case["M"] * (case["K"] * (size + 1) + 8), "flops": 2 * case["M"] * case["K"]}
    if case["op"] == "swiglu":
        return {"bytes": case["M"] * (case["K"] * 5 + 8), "flops": 6 * case["M"] * case["K"]}
    K, N = case["K"], case["N"]
    per_channel = 2 + (1 if case["asym"] else 0) + (2 if case["bias"] else 0)
    if case["op"] == "linear":
        M = case["M"]
        return {"bytes": K * N + per_channel * N + M * (K + 8) + 2 * M * N, "flops": 2 * M * K * N}
    rows = case["T"] - case["behind"]
    # an expert without rows needs no weight: the number that even shares leave with some
    experts = case["E"] * (1 - (1 - 1 / case["E"]) ** rows)
    return {"bytes": int(experts * (K * N + per_channel * N)) + rows * (K + 8) + 2 * rows * N + 4 * (case["E"] + 1),
            "flops": 2 * rows * K * N}


# ---------------------------------------------------------------- inputs
def _activations(g, M, K, dtype):
    """N(0, 1) with a few wide features, as after a norm layer."""
    x = torch.randn((M, K), generator=g, device="cuda")
    wide = torch.rand((K,), generator=g, device="cuda") < 0.002
    return (x * (1 + 9 * wide)).to(dtype)


def _codes(g, K, N, asym):
    """Codes as a channel-wise quantizer leaves them: the largest of some
    thousand normal values on the last level."""
    q = torch.randn((K, N), generator=g, device="cuda") * (127 / 4.2)
    if asym:
        return (q + 6).round_().clamp_(-128, 127).to(torch.int8)
    return q.round_().clamp_(-127, 127).to(torch.int8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"op": case["op"]}
    if case["op"] == "tokens":
        s["X"] = _activations(g, case["M"], case["K"], getattr(torch, case["dtype"]))
        return s
    if case["op"] == "swiglu":
        # the first product's output, gate half then up half
        s["H"] = (1.5 * torch.randn((case["M"], 2 * case["K"]), generator=g, device="cuda")).half()
        return s
    K, N = case["K"], case["N"]
    E = case.get("E", 1)
    rows = case["M"] if case["op"] == "linear" else case["T"]
    s["q"], s["xs"], s["sums"] = _plain_quantize(_activations(g, rows, K, torch.float16).float())
    s["w"] = torch.empty((E, K, N), dtype=torch.int8, device="cuda")
    for e in range(E):
        s["w"][e] = _codes(g, K, N, case["asym"])
    s["scales"] = ((0.5 + torch.rand((E, N), generator=g, device="cuda")) * (0.09 / 127)).half()
    s["zeros"] = (torch.randint(-12, 25, (E, N), generator=g, device="cuda").to(torch.int8) if case["asym"] else None)
    s["bias"] = (0.1 * torch.randn((E, N), generator=g, device="cuda")).half() if case["bias"] else None
    if K % 16:   # the library wants rows of codes on 16-byte boundaries
        wide = torch.zeros((rows, (K + 15) // 16 * 16), dtype=torch.int8, device="cuda")
        wide[:, :K] = s["q"]
        s["q"] = wide[:, :K]
    if case["op"] == "grouped":
        # the router's choice: expert e with weight exp(skew * normal)
        share = torch.exp(case["skew"] * torch.randn((E,), generator=g, device="cuda"))
        if E > 8:
            share[E // 3] = 0.0   # an expert that no token chose
        chosen = torch.multinomial(share, rows - case["behind"], replacement=True, generator=g)
        counts = torch.bincount(chosen, minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["capacity"] = int(counts.max())   # the plain form's padded group length
        s["Y"] = torch.full((rows, N), 0.5, dtype=torch.float16, device="cuda")
    if own:
        import int8_weight_only_b200 as w8
        s["packed"] = torch.stack([w8.prepack(s["w"][e]) for e in range(E)])
    if case["op"] == "linear":
        for k in ("w", "scales", "zeros", "bias", "packed"):
            s[k] = s[k][0] if s.get(k) is not None else None
    return s


# ---------------------------------------------------------------- one pass
def _plain_quantize(x):
    """Codes, scales and sums of codes of fp32 rows: every step one IEEE fp32 operation."""
    scale = x.abs().amax(1, keepdim=True) / torch.full((1, 1), 127.0, device=x.device)
    q = torch.where(scale > 0, torch.clamp(torch.round(x / scale), -127, 127), 0.0)
    return q.to(torch.int8), scale[:, 0], q.sum(1, dtype=torch.int64).to(torch.int32)


def _values(q, scale, dtype):
    """What the codes stand for, in the activations' type."""
    out = torch.empty(q.shape, dtype=dtype, device=q.device)
    return torch.mul(q, scale[:, None], out=out)


def _plain_weight(w, zeros):
    w = w.float()
    return w if zeros is None else w - zeros.float().unsqueeze(-2)


def _plain_scale(acc, xs, scales, bias):
    y = acc * xs.unsqueeze(-1) * scales.float().unsqueeze(-2)
    return y if bias is None else y + bias.float().unsqueeze(-2)


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_plain(s):
    if s["op"] == "tokens":
        q, scale, sums = _plain_quantize(s["X"].float())
        return _values(q, scale, s["X"].dtype), scale, sums
    if s["op"] == "swiglu":
        gate, up = s["H"].float().chunk(2, dim=1)
        q, scale, sums = _plain_quantize(gate / (1 + torch.exp(-gate)) * up)
        return _values(q, scale, torch.float16), scale, sums
    if s["op"] == "linear":
        acc = s["q"].float() @ _plain_weight(s["w"], s["zeros"])
        return _plain_scale(acc, s["xs"], s["scales"], s["bias"]).half()
    # every group padded to the longest one, then one batched product
    T, first, last = s["q"].shape[0], s["offsets"][:-1].long(), s["offsets"][1:].long()
    row = first[:, None] + torch.arange(s["capacity"], device="cuda")
    row = torch.minimum(row, row.new_full((), T - 1))
    acc = torch.bmm(s["q"].float()[row], _plain_weight(s["w"], s["zeros"]))
    y = _plain_scale(acc, s["xs"][row], s["scales"], s["bias"]).half()
    at = torch.arange(T, device="cuda")
    expert = torch.clamp(torch.searchsorted(last, at, right=True), max=last.numel() - 1)
    place = torch.clamp(at - first[expert], 0, s["capacity"] - 1)
    s["Y"].copy_(torch.where((at < last[-1])[:, None], y[expert, place], s["Y"]))
    return s["Y"]


def _run_own(s):
    import int8_weight_only_b200 as w8
    if s["op"] == "tokens":
        q, scale, sums = w8.quantize_tokens(s["X"])
        return _values(q, scale, s["X"].dtype), scale, sums
    if s["op"] == "swiglu":
        q, scale, sums = w8.swiglu_quantize_tokens(s["H"])
        return _values(q, scale, torch.float16), scale, sums
    if s["op"] == "linear":
        return w8.linear_w8a8(s["q"], s["xs"], s["sums"], s["packed"], s["scales"], bias=s["bias"], zeros=s["zeros"])
    return w8.linear_w8a8_grouped(s["q"], s["xs"], s["sums"], s["offsets"], s["packed"], s["scales"], bias=s["bias"],
                                  zeros=s["zeros"], out=s["Y"])


# ---------------------------------------------------------------- the definition, in 64 bits
def _exact_rows(x, scale):
    """Codes by the definition: the quotient rounded to fp32, then to the
    nearest integer, halves to even."""
    ratio = (x / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]).float().double()
    return torch.clamp(torch.round(ratio), -127, 127) * (scale > 0)[:, None]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("tokens", "swiglu"):
        if case["op"] == "tokens":
            x = s["X"].double()
        else:
            H = s["H"].double()
            K = case["K"]
            x = H[:, :K] * torch.sigmoid(H[:, :K]) * H[:, K:]
        scale = (x.abs().max(dim=1).values / 127).float().double()
        q = _exact_rows(x, scale)
        return q * scale[:, None], scale, q.sum(1).long()
    x = s["q"].double() * s["xs"].double()[:, None]
    if case["op"] == "linear":
        w = s["w"].double()
        if case["asym"]:
            w -= s["zeros"].double()
        y = x @ (w * s["scales"].double())
        return y + s["bias"].double() if case["bias"] else y
    y = s["Y"].double()
    at = s["offsets"].tolist()
    for e in range(case["E"]):
        if at[e + 1] > at[e]:
            w = s["w"][e].double()
            if case["asym"]:
                w -= s["zeros"][e].double()
            y[at[e]:at[e + 1]] = x[at[e]:at[e + 1]] @ (w * s["scales"][e].double())
            if case["bias"]:
                y[at[e]:at[e + 1]] += s["bias"][e].double()
    return y
