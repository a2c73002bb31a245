"""Cases that measure the 4-bit linears with scales per group and the sampler of tokens.

`run` computes an operator either from elementary torch operations (own = False) or through the library's entry
points (own = True); `exact` gives the same values from the definition in 64 bits.

A 4-bit weight holds two codes per byte, low nibble first, and is (code - zero) * scale with one f16 scale per group
of inputs; the zero point is 8 everywhere, a 4-bit code per group (packed like the weights), or an f16 per group.

The sampler draws a token of each row of logits: temperature, then min-p, top-k and top-p, each of which leaves the
first tokens in descending order of their logits (equal logits: the lower token first), and the first token of that
order whose cumulative probability exceeds the given random number.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
DTYPES = {"bf16": BF16, "f32": F32}
MOST_WEIGHTS = 1 << 28             # of a drawn linear; the largest listed one has twice as many
MOST_LOGITS = 1 << 24              # of a drawn batch; the largest listed one has twice as many


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _linear(m, k, n, group, zero, act="none", gated=False, bias=False, residual="", out="bf16"):
    """n counts the output columns; a gated layer's weight has 2 n rows."""
    return {"op": "linear", "m": m, "k": k, "n": n, "group": group, "zero": zero, "act": act, "gated": gated,
            "bias": bias, "residual": residual, "out": out}


def _sample(rows, vocab, dtype="f32", temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, mixed=False, masked=0.0, pad=0):
    """pad: columns behind the vocabulary that the rows of logits have; masked: the part of the tokens that a row
    rules out; mixed: every row has settings of its own, some rows take their largest logit."""
    return {"op": "sample", "rows": rows, "vocab": vocab, "dtype": dtype, "temperature": temperature, "top_k": top_k,
            "top_p": top_p, "min_p": min_p, "mixed": mixed, "masked": masked, "pad": pad}


def listed():
    return [
        # one token through a text model's gated layer: latency and the read of the weight
        dict(_linear(1, 2560, 9728, 64, "f16", act="silu", gated=True), name="token gated g64"),
        # and back onto the residual stream, symmetric weights with a scale per 32
        dict(_linear(1, 9728, 2560, 32, "none", residual="bf16"), name="token down g32 symmetric"),
        # a decode batch through the attention's fused projection, with its bias
        dict(_linear(13, 2560, 6144, 64, "codes", bias=True), name="batch of 13 g64"),
        # one token's logits over an odd vocabulary: the largest read of a single token
        dict(_linear(1, 2560, 128009, 64, "f16", out="f32"), name="token logits g64"),
        # a decode batch's logits
        dict(_linear(32, 4096, 128009, 32, "codes", out="f32"), name="batch logits g32"),
        # a larger batch, symmetric weights with a scale per 128
        dict(_linear(61, 2560, 9728, 128, "none", act="gelu_tanh"), name="batch of 61 g128 symmetric"),
        # one token out of a small vocabulary: latency
        dict(_sample(1, 4099, top_k=50), name="sample token small"),
        # one token, the usual settings
        dict(_sample(1, 128009, temperature=0.8, top_k=40, top_p=0.95), name="sample token"),
        # a batch from the whole distribution
        dict(_sample(32, 128009, temperature=0.9), name="sample batch"),
        # a batch with a nucleus, logits in 16 bits (ties), rows padded
        dict(_sample(64, 128009, dtype="bf16", top_p=0.9, pad=55), name="sample batch nucleus bf16"),
        # a large batch with a lower bound relative to the best token
        dict(_sample(256, 128009, temperature=1.2, min_p=0.02), name="sample large batch min-p"),
        # requests with settings of their own, a grammar that rules most tokens out
        dict(_sample(96, 50021, mixed=True, masked=0.7), name="sample mixed requests"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        group = rng.choice([32, 32, 64, 64, 128, 256])
        zero = rng.choice(["none", "codes"] if group == 128 else ["none", "codes", "f16"])
        k = group * _log(rng, max(1, 256 // group), 9728 // group)
        gated = rng.random() < 0.3
        most = min(65536, MOST_WEIGHTS // (k * (2 if gated else 1)))
        return _linear(_log(rng, 1, 64), k, _log(rng, 64, most), group, zero,
                       act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), gated=gated,
                       bias=rng.random() < 0.3, residual=rng.choice(["", "bf16", "f32"]),
                       out=rng.choice(["bf16", "f32"]))
    vocab = _log(rng, 100, 131072)
    return _sample(_log(rng, 1, min(512, MOST_LOGITS // vocab)), vocab, dtype=rng.choice(["f32", "bf16"]),
                   temperature=round(rng.uniform(0.4, 1.5), 2), top_k=rng.choice([0, 1, _log(rng, 2, vocab)]),
                   top_p=rng.choice([1.0, round(rng.uniform(0.2, 0.99), 2)]),
                   min_p=rng.choice([0.0, 0.0, round(rng.uniform(0.001, 0.2), 3)]), mixed=rng.random() < 0.25,
                   masked=rng.choice([0.0, 0.5]), pad=rng.choice([0, rng.randint(1, 64)]))


def _wrows(case):
    return case["n"] * (2 if case["gated"] else 1)


def work(case):
    size = {"bf16": 2, "f32": 4, "": 0}
    if case["op"] == "linear":
        m, k, n, w, groups = case["m"], case["k"], case["n"], _wrows(case), case["k"] // case["group"]
        zero = {"none": 0, "codes": (groups + 1) // 2, "f16": 2 * groups}[case["zero"]]
        return {"bytes": w * (k // 2 + 2 * groups + zero) + 2 * m * k + (4 * w if case["bias"] else 0)
                + m * n * (size[case["out"]] + size[case["residual"]]),
                "flops": 2 * m * w * k}
    b, v = case["rows"], case["vocab"]
    return {"bytes": b * (v * size[case["dtype"]] + 12 + (16 if case["mixed"] else 0)), "flops": 3 * b * v}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=DEV)

    def uniform(*shape):
        return torch.rand(shape, generator=g, device=DEV)

    def choice(values, n, dtype):
        at = torch.randint(0, len(values), (n,), generator=g, device=DEV)
        return torch.tensor(values, device=DEV, dtype=dtype)[at]

    s = {"case": case}
    if case["op"] == "linear":
        m, k, n, w, groups = case["m"], case["k"], case["n"], _wrows(case), case["k"] // case["group"]
        s["x"] = normal(m, k).to(BF16)
        s["packed"] = torch.randint(0, 256, (w, k // 2), generator=g, device=DEV, dtype=torch.uint8)
        s["scale"] = (normal(w, groups).abs() * 0.02).half()
        s["zero"] = None
        if case["zero"] == "f16":
            s["zero"] = (uniform(w, groups) * 15).half()
        elif case["zero"] == "codes":
            s["zero"] = torch.randint(0, 256, (w, (groups + 1) // 2), generator=g, device=DEV, dtype=torch.uint8)
        s["bias"] = normal(w) * 0.2 if case["bias"] else None
        s["residual"] = normal(m, n).to(DTYPES[case["residual"]]) if case["residual"] else None
        return s
    b, v = case["rows"], case["vocab"]
    logits = normal(b, v + case["pad"]) * 2.5 + normal(v + case["pad"])       # some tokens are likelier everywhere
    logits[uniform(b, v + case["pad"]) < 3e-4] += 8                           # the few that fit
    if case["masked"]:
        logits[uniform(b, v + case["pad"]) < case["masked"]] = -math.inf
    s["logits"] = logits.to(DTYPES[case["dtype"]])[:, :v]
    s["u"] = uniform(b)
    s["settings"] = {key: case[key] for key in ("temperature", "top_k", "top_p", "min_p")}
    if case["mixed"]:
        s["settings"] = {"temperature": choice([0.0, 0.6, 0.8, 1.0, 1.3], b, F32),
                         "top_k": choice([0, 0, 1, 20, 1000], b, torch.int32),
                         "top_p": choice([1.0, 0.95, 0.8, 0.5], b, F32),
                         "min_p": choice([0.0, 0.0, 0.05], b, F32)}
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _nibbles(packed):
    return torch.stack([packed & 15, packed >> 4], dim=-1).flatten(1)


def _run_linear(s):
    c = s["case"]
    groups = c["k"] // c["group"]
    q = _nibbles(s["packed"]).view(-1, groups, c["group"]).float()
    zero = s["zero"]
    if zero is None:
        q = q - 8
    else:
        q = q - (zero.float() if c["zero"] == "f16" else _nibbles(zero)[:, :groups].float()).unsqueeze(-1)
    v = s["x"].float() @ (q * s["scale"].float().unsqueeze(-1)).flatten(1).t()
    if s["bias"] is not None:
        v = v + s["bias"]
    a = v[:, :c["n"]] if c["gated"] else v
    if c["act"] == "relu":
        a = a.clamp(min=0)
    elif c["act"] == "gelu":
        a = 0.5 * a * (1 + torch.erf(a * math.sqrt(0.5)))
    elif c["act"] == "gelu_tanh":
        a = 0.5 * a * (1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a * a * a)))
    elif c["act"] == "silu":
        a = a / (1 + torch.exp(-a))
    if c["gated"]:
        a = a * v[:, c["n"]:]
    if s["residual"] is not None:
        a = a + s["residual"].float()
    return a.to(DTYPES[c["out"]])


def _column(value, like):
    """A setting per row, as a column."""
    if not isinstance(value, torch.Tensor):
        value = torch.full((like.shape[0],), value, device=DEV)
    return value.unsqueeze(1)


def _run_sample(s):
    # in 64 bits: a draw or a nucleus that ends next to a border must not depend on rounding
    v = s["logits"].float()
    v = torch.where(v > -math.inf, v, -math.inf)                       # a NaN is masked
    ranked, token = v.sort(dim=1, descending=True, stable=True)        # ties: the lower token first
    st = s["settings"]
    temperature = _column(st["temperature"], v).double()
    top_k, top_p, min_p = (_column(st[k], v).float() if k != "top_k" else _column(st[k], v)
                           for k in ("top_k", "top_p", "min_p"))
    rank = torch.arange(v.shape[1], device=DEV)
    best = ranked[:, :1]
    p = torch.exp((ranked.double() - best.double()) / temperature)
    p = torch.where(ranked == best, 1.0, p).nan_to_num(0.0)
    p = torch.where(ranked == -math.inf, 0.0, p)
    keep = (p >= min_p.double()) & ((rank < top_k) | (top_k <= 0)) | (rank == 0)
    p = torch.where(keep, p, 0.0)
    c = p.cumsum(1)
    keep = (c - p < top_p.double() * c[:, -1:]) | (top_p >= 1) | (rank == 0)
    p = torch.where(keep, p, 0.0)
    c = p.cumsum(1)
    total = c[:, -1:]
    at = (c <= s["u"].double().unsqueeze(1) * total).sum(1, keepdim=True)
    at = torch.minimum(at, (p > 0).sum(1, keepdim=True) - 1).clamp(min=0)
    at = torch.where(temperature > 0, at, 0)
    prob = torch.where(temperature > 0, p.gather(1, at) / total, 1.0)
    live = best > -math.inf
    return (torch.where(live, token.gather(1, at), -1).squeeze(1).int(),
            torch.where(live, prob, 0.0).squeeze(1).float())


def run(state):
    c = state["case"]
    if not own:
        return _run_linear(state) if c["op"] == "linear" else _run_sample(state)
    import ternary_weight_quantized_q2_amd as q2
    if c["op"] == "linear":
        return q2.q4_matvec(state["x"], state["packed"], state["scale"], state["zero"], bias=state["bias"],
                             activation=c["act"], gated=c["gated"], residual=state["residual"],
                             out_dtype=DTYPES[c["out"]])
    return tuple(q2.q2_sample(state["logits"], state["u"], **state["settings"]))


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _exact_linear(case, s):
    codes = torch.tensor([[byte % 16, byte // 16] for byte in range(256)], dtype=F64, device=DEV)
    x, group, groups = s["x"].double(), case["group"], case["k"] // case["group"]
    parts = []
    for lo in range(0, _wrows(case), 16384):                           # a part of the weight's rows at a time
        rows = slice(lo, lo + 16384)
        w = codes[s["packed"][rows].int()].flatten(1)
        zero = 8.0
        if case["zero"] == "codes":
            zero = codes[s["zero"][rows].int()].flatten(1)[:, :groups].repeat_interleave(group, dim=1)
        elif case["zero"] == "f16":
            zero = s["zero"][rows].double().repeat_interleave(group, dim=1)
        parts.append(x.matmul((w - zero).mul_(s["scale"][rows].double().repeat_interleave(group, dim=1)).mT))
    z = torch.cat(parts, dim=1)
    if case["bias"]:
        z += s["bias"].double()
    a, b = z.chunk(2, dim=1) if case["gated"] else (z, 1.0)
    if case["act"] == "relu":
        a = torch.maximum(a, torch.zeros_like(a))
    elif case["act"] == "silu":
        a = a * torch.special.expit(a)
    elif case["act"] == "gelu":
        a = a * torch.special.ndtr(a)
    elif case["act"] == "gelu_tanh":                                   # (1 + tanh(t / 2)) / 2 is the logistic function
        a = a * torch.special.expit(math.sqrt(8 / math.pi) * (a + 0.044715 * a ** 3))
    y = a * b
    return y + s["residual"].double() if case["residual"] else y


def _exact_row(v, u, temperature, top_k, top_p, min_p):
    """(token, probability) of one row by its distinct logits, each with the number of tokens that have it."""
    value, count = torch.unique(v[v > -math.inf], return_counts=True)
    if value.numel() == 0:
        return -1, 0.0
    value, count = value.flip(0), count.flip(0)
    if not temperature > 0:
        return int((v == value[0]).nonzero()[0]), 1.0
    w = torch.cat([torch.ones_like(value[:1]), torch.exp((value[1:] - value[0]) / temperature)])
    if min_p > 0:
        w, count = w[:max(1, int((w >= min_p).sum()))], count[:max(1, int((w >= min_p).sum()))]
        if min_p > 1:
            count = torch.ones_like(count)
    if top_k > 0:
        before = count.cumsum(0) - count
        count = (top_k - before).clamp(min=0).minimum(count)
    if top_p < 1:
        most = top_p * (w * count).sum()
        before = (w * count).cumsum(0) - w * count
        count = torch.ceil((most - before) / w).clamp(min=0).nan_to_num(0.0).minimum(count.double())
        count[0] = count[0].clamp(min=1)
    sums = (w * count).cumsum(0)
    target = u * sums[-1]
    at = min(int((sums <= target).sum()), int(((w > 0) & (count > 0)).sum()) - 1)
    within = int(((target - (sums[at - 1] if at else 0.0)) / w[at]).floor())
    within = min(max(within, 0), int(count[at]) - 1)
    return int((v == value[at]).nonzero()[within]), float(w[at] / sums[-1])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        return _exact_linear(case, s)

    def of(row, name):
        t = s["settings"][name]
        return t[row].item() if isinstance(t, torch.Tensor) else torch.tensor(t, dtype=F32).item()

    drawn = [_exact_row(s["logits"][i].double(), s["u"][i].item(),
                        *(of(i, name) for name in ("temperature", "top_k", "top_p", "min_p")))
             for i in range(case["rows"])]
    return (torch.tensor([t for t, _ in drawn], dtype=torch.int32, device=DEV),
            torch.tensor([p for _, p in drawn], dtype=F64, device=DEV))
