"""Cases that measure the fused and grouped linears, the router and the combination of the experts' outputs.

`run` computes an operator either from elementary torch operations in 32 bits (own = False) or through the
library's entry points (own = True); `exact` gives the same values from the definition in 64 bits.

Weights are packed as the library defines them: Q2_0 holds four 2-bit codes per byte, lowest pair first, a weight
is (code - 1) * scale with one f16 scale per 128 inputs; the 4-bit format holds two codes per byte, low nibble
first, a weight is (code - zero) * scale.
"""
import math

import torch

own = False

BLOCK = 128
MOST_PRODUCTS = 1 << 37            # of a drawn case, less than the largest listed case has
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "f32": F32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _fused(m, k, n, fmt="q2", act="none", gated=False, bias=False, gate=False, residual="", out="bf16", rank=0):
    """n counts the output columns; a gated layer's weight has 2 n rows."""
    return {"op": "fused", "m": m, "k": k, "n": n, "fmt": fmt, "act": act, "gated": gated, "bias": bias, "gate": gate,
            "residual": residual, "out": out, "rank": rank}


def _grouped(tokens, top, experts, k, n, fmt="q2", act="none", gated=False, bias=False, gather=False, out="bf16"):
    """tokens * top rows over the experts; gather reads a token's row through an index, as the first of an
    expert's two layers does, the second reads its rows in place."""
    return {"op": "grouped", "tokens": tokens, "top": top, "experts": experts, "k": k, "n": n, "fmt": fmt, "act": act,
            "gated": gated, "bias": bias, "gather": gather, "out": out}


def _route(tokens, top, experts, dtype="f32", renorm=True, padded=0.0):
    return {"op": "route", "tokens": tokens, "top": top, "experts": experts, "dtype": dtype, "renorm": renorm,
            "padded": padded}


def _combine(tokens, top, n, dtype="bf16", residual="bf16", out="bf16", dropped=0.0):
    return {"op": "combine", "tokens": tokens, "top": top, "n": n, "dtype": dtype, "residual": residual, "out": out,
            "dropped": dropped}


def listed():
    return [
        # one token through a text model's gated layer (2560 -> 9728): latency and the read of the weight
        dict(_fused(1, 2560, 9728, act="silu", gated=True), name="fused token gated"),
        # a 128-token prompt through the same layer in the 4-bit format
        dict(_fused(128, 2560, 9728, fmt="q4", act="silu", gated=True), name="fused prompt gated 4-bit"),
        # an image transformer's first MLP layer, 1024 image and 512 text rows
        dict(_fused(1536, 4096, 12288, act="gelu_tanh", bias=True), name="fused image mlp in"),
        # its second one with the rank-32 branch, the block's gate and the residual stream in 32 bits, several images
        # whose row count is no multiple of any tile
        dict(_fused(4093, 12288, 4096, bias=True, gate=True, residual="f32", out="f32", rank=32),
             name="fused image mlp out"),
        # one token through its eight experts' gated layers
        dict(_grouped(1, 8, 64, 2048, 1024, act="silu", gated=True, gather=True), name="grouped token gated"),
        # a decode batch: a few rows for each expert, 4-bit, with a bias
        dict(_grouped(23, 4, 32, 2560, 1408, fmt="q4", act="relu", bias=True, gather=True),
             name="grouped batch 4-bit"),
        # a prompt's rows through the experts' gated layers, ragged counts
        dict(_grouped(2048, 4, 32, 2048, 1408, act="silu", gated=True, gather=True), name="grouped prompt gated"),
        # and back, the rows in place
        dict(_grouped(2048, 4, 32, 1408, 2048), name="grouped prompt down"),
        # one token's routing: latency alone
        dict(_route(1, 8, 64), name="route token"),
        # a large batch with padding tokens, logits in 16 bits (ties)
        dict(_route(16384, 8, 128, dtype="bf16", padded=0.1), name="route batch"),
        # one token's experts summed onto the residual stream
        dict(_combine(1, 8, 2048), name="combine token"),
        # a prompt's
        dict(_combine(8192, 4, 2048, dropped=0.05), name="combine prompt"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fused", "fused", "grouped", "grouped", "route", "combine"])
    acts = ["none", "relu", "gelu", "gelu_tanh", "silu"]
    if op == "fused":
        k = BLOCK * _log(rng, 4, 96)
        n = _log(rng, 200, 12288)
        gated = rng.random() < 0.4
        most = min(4096, MOST_PRODUCTS // (k * n * (2 if gated else 1)))
        fmt = rng.choice(["q2", "q2", "q4"])
        return _fused(_log(rng, 1, most), k, n, fmt=fmt, act=rng.choice(acts), gated=gated, bias=rng.random() < 0.5,
                      gate=rng.random() < 0.3, residual=rng.choice(["", "bf16", "f32"]),
                      out=rng.choice(["bf16", "f32"]), rank=rng.choice([0, _log(rng, 4, 64)]) if fmt == "q2" else 0)
    if op == "grouped":
        experts = _log(rng, 4, 128)
        top = rng.randint(1, min(8, experts))
        k, n, gated = BLOCK * _log(rng, 4, 20), _log(rng, 100, 2048), rng.random() < 0.5
        most = min(4096, MOST_PRODUCTS // (top * k * n * (2 if gated else 1)))
        return _grouped(_log(rng, 1, most), top, experts, k, n, fmt=rng.choice(["q2", "q2", "q4"]),
                        act=rng.choice(acts), gated=gated, bias=rng.random() < 0.3, gather=rng.random() < 0.5,
                        out=rng.choice(["bf16", "f32"]))
    if op == "route":
        experts = _log(rng, 4, 256)
        return _route(_log(rng, 1, 16384), rng.randint(1, min(8, experts)), experts, dtype=rng.choice(["f32", "bf16"]),
                      renorm=rng.random() < 0.5, padded=rng.choice([0.0, 0.2]))
    return _combine(_log(rng, 1, 8192), rng.randint(1, 8), _log(rng, 64, 4096), dtype=rng.choice(["bf16", "f32"]),
                    residual=rng.choice(["", "bf16", "f32"]), out=rng.choice(["bf16", "f32"]),
                    dropped=rng.choice([0.0, 0.1]))


def _wrows(case):
    return case["n"] * (2 if case["gated"] else 1)


def work(case):
    size = {"bf16": 2, "f32": 4, "": 0}
    if case["op"] in ("fused", "grouped"):
        k, n, w = case["k"], case["n"], _wrows(case)
        per = (BLOCK // 4 + 2) if case["fmt"] == "q2" else (BLOCK // 2 + 4)
        weight = w * (k // BLOCK) * per + (4 * w if case["bias"] else 0)
        if case["op"] == "fused":
            m, r = case["m"], case["rank"]
            return {"bytes": weight + 2 * m * k + m * n * (size[case["out"]] + size[case["residual"]])
                    + 2 * r * (k + w) + (4 * n if case["gate"] else 0),
                    "flops": 2 * m * w * k + 2 * m * r * (k + w)}
        t, e = case["tokens"], case["experts"]
        rows = t * case["top"]
        used = e * (1 - (1 - case["top"] / e) ** t)          # experts that some token chose
        x_rows = t if case["gather"] else rows
        return {"bytes": int(weight * used) + 2 * x_rows * k + rows * n * size[case["out"]] + 4 * (e + 1)
                + (4 * rows if case["gather"] else 0),
                "flops": 2 * rows * w * k}
    t, j = case["tokens"], case["top"]
    if case["op"] == "route":
        e = case["experts"]
        return {"bytes": t * e * size[case["dtype"]] + 16 * t * j + 4 * (e + 1), "flops": 3 * t * e + t * e * j}
    n = case["n"]
    return {"bytes": t * j * (n * size[case["dtype"]] + 8) + t * n * (size[case["residual"]] + size[case["out"]]),
            "flops": 2 * t * j * n}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _weights(g, fmt, shape, k):
    """Packed weight of `shape` rows (a tuple: rows, or experts and rows) and k inputs, as a loader leaves it."""
    blocks = (*shape, k // BLOCK)
    scale = (torch.randn(blocks, generator=g, device=DEV).abs() * 0.02).half()
    if fmt == "q2":
        # four 2-bit codes drawn at once: a byte out of the 81 whose codes are all below 3
        digits = torch.randint(0, 81, (*shape, k // 4), generator=g, device=DEV, dtype=torch.int32)
        packed = (digits % 3) | (digits // 3 % 3) << 2 | (digits // 9 % 3) << 4 | (digits // 27) << 6
        return [packed.to(torch.uint8), scale]
    packed = torch.randint(0, 256, (*shape, k // 2), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
    zero = (torch.rand(blocks, generator=g, device=DEV) * 15).half()
    return [packed, scale, zero]


def _vector(g, n, std):
    return torch.randn(n, generator=g, device=DEV) * std


def _logits(g, t, e):
    """Router logits: experts are not equally popular."""
    return torch.randn((t, e), generator=g, device=DEV) + torch.randn(e, generator=g, device=DEV) * 0.5


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] == "fused":
        m, k, n, w = case["m"], case["k"], case["n"], _wrows(case)
        s["x"] = torch.randn((m, k), generator=g, device=DEV).to(BF16)
        s["w"] = _weights(g, case["fmt"], (w,), k)
        s["bias"] = _vector(g, w, 0.2) if case["bias"] else None
        s["gate"] = _vector(g, n, 1.0) if case["gate"] else None
        s["residual"] = (torch.randn((m, n), generator=g, device=DEV).to(DTYPES[case["residual"]])
                         if case["residual"] else None)
        r = case["rank"]
        s["A"] = _vector(g, (r, k), 0.01).half() if r else None
        s["B"] = _vector(g, (w, r), 0.01).half() if r else None
    elif case["op"] == "grouped":
        t, top, e, k, w = case["tokens"], case["top"], case["experts"], case["k"], _wrows(case)
        rows = t * top
        chosen = _logits(g, t, e).topk(top).indices.flatten()
        order = chosen.argsort(stable=True)
        s["offsets"] = torch.searchsorted(chosen[order], torch.arange(e + 1, device=DEV)).int()
        s["index"] = (order // top).int() if case["gather"] else None
        s["x"] = torch.randn((t if case["gather"] else rows, k), generator=g, device=DEV).to(BF16)
        s["w"] = _weights(g, case["fmt"], (e, w), k)
        s["bias"] = _vector(g, (e, w), 0.2) if case["bias"] else None
    elif case["op"] == "route":
        t, e = case["tokens"], case["experts"]
        logits = _logits(g, t, e)
        if case["padded"]:                                    # padding tokens: every expert masked
            logits[torch.rand(t, generator=g, device=DEV) < case["padded"]] = -math.inf
        s["logits"] = logits.to(DTYPES[case["dtype"]])
    else:
        t, top, n = case["tokens"], case["top"], case["n"]
        rows = t * top
        s["z"] = torch.randn((rows, n), generator=g, device=DEV).to(DTYPES[case["dtype"]])
        slot = torch.rand(rows, generator=g, device=DEV).argsort().int()
        if case["dropped"]:
            slot[torch.rand(rows, generator=g, device=DEV) < case["dropped"]] = -1
        s["slot"] = slot.view(t, top)
        s["weight"] = torch.rand((t, top), generator=g, device=DEV)
        s["residual"] = (torch.randn((t, n), generator=g, device=DEV).to(DTYPES[case["residual"]])
                         if case["residual"] else None)
    return s


# ---------------------------------------------------------------------------
# plain forms, in 32 bits
# ---------------------------------------------------------------------------

def _dequant(w, fmt):
    """float32 weights [..., rows, inputs] of a packed weight."""
    packed, scale = w[0], w[1].float().unsqueeze(-1)
    if fmt == "q2":
        q = (packed.unsqueeze(-1) >> torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device=DEV)) & 3
    else:
        q = (packed.unsqueeze(-1) >> torch.tensor([0, 4], dtype=torch.uint8, device=DEV)) & 15
    q = q.view(*scale.shape[:-1], BLOCK).float()
    zero = 1.0 if fmt == "q2" else w[2].float().unsqueeze(-1)
    return ((q - zero) * scale).flatten(-2)


def _activate(name, v):
    if name == "relu":
        return v.clamp(min=0)
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    if name == "silu":
        return v / (1 + torch.exp(-v))
    return v


def _epilogue(case, v):
    if not case["gated"]:
        return _activate(case["act"], v)
    return _activate(case["act"], v[..., :case["n"]]) * v[..., case["n"]:]


def _run_fused(s):
    c = s["case"]
    x = s["x"].float()
    v = x @ _dequant(s["w"], c["fmt"]).t()
    if s["A"] is not None:
        v = v + (x @ s["A"].float().t()) @ s["B"].float().t()
    if s["bias"] is not None:
        v = v + s["bias"]
    v = _epilogue(c, v)
    if s["gate"] is not None:
        v = v * s["gate"]
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v.to(DTYPES[c["out"]])


def _run_grouped(s):
    c = s["case"]
    x = (s["x"] if s["index"] is None else s["x"][s["index"].long()]).float()
    rows, e = x.shape[0], c["experts"]
    pos = torch.arange(rows, device=DEV)
    expert = torch.searchsorted(s["offsets"][1:].contiguous(), pos, right=True)
    if rows <= e:
        # few rows: the weight of each row's expert
        w = _dequant([t[expert] for t in s["w"]], c["fmt"])
        v = torch.bmm(w, x.unsqueeze(-1)).squeeze(-1)
    else:
        # the rows of each expert padded to the longest group, one batched product
        first = s["offsets"].long()
        most = int((first[1:] - first[:-1]).max())
        padded = torch.zeros((e, most, c["k"]), device=DEV)
        padded[expert, pos - first[expert]] = x
        w = _dequant(s["w"], c["fmt"])
        v = torch.bmm(padded, w.transpose(1, 2))[expert, pos - first[expert]]
    if s["bias"] is not None:
        v = v + s["bias"][expert]
    return _epilogue(c, v).to(DTYPES[c["out"]])


def _run_route(s):
    c = s["case"]
    top, e = c["top"], c["experts"]
    v = s["logits"].float()
    ranked, expert = v.sort(dim=1, descending=True, stable=True)       # ties: the lowest expert first
    p = torch.exp(ranked - ranked[:, :1])
    p = torch.where(ranked == -math.inf, 0.0, p)                       # masked experts, whole masked tokens too
    total = p[:, :top].sum(1, keepdim=True) if c["renorm"] else p.sum(1, keepdim=True)
    live = ranked[:, :top] != -math.inf
    weight = torch.where(live, p[:, :top] / total, 0.0)
    expert = torch.where(live, expert[:, :top], -1)
    # rows sorted by expert, then by token; choices of masked experts get no row
    flat = expert.flatten()
    key = torch.where(flat < 0, e, flat)
    key, order = key.sort(stable=True)
    offsets = torch.searchsorted(key, torch.arange(e + 1, device=DEV))
    token = torch.where(key < e, order // top, -1)
    slot = torch.empty_like(order)
    slot[order] = torch.where(key < e, torch.arange(flat.numel(), device=DEV), -1)
    return expert.int(), weight, offsets.int(), token.int(), slot.view(-1, top).int()


def _run_combine(s):
    live = s["slot"] >= 0
    z = s["z"][s["slot"].clamp(min=0).long()].float()
    y = torch.where(live.unsqueeze(-1), z * s["weight"].unsqueeze(-1), 0.0).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DTYPES[s["case"]["out"]])


def run(state):
    c = state["case"]
    op = c["op"]
    if not own:
        return {"fused": _run_fused, "grouped": _run_grouped, "route": _run_route, "combine": _run_combine}[op](state)
    import ternary_weight_quantized_q2_amd as q2
    if op == "fused":
        extra = dict(bias=state["bias"], activation=c["act"], gated=c["gated"], gate=state["gate"],
                     residual=state["residual"], out_dtype=DTYPES[c["out"]])
        if c["fmt"] == "q4":
            return q2.q4_linear_fused(state["x"], *state["w"], **extra)
        return q2.q2_linear_fused(state["x"], *state["w"], A=state["A"], B=state["B"], **extra)
    if op == "grouped":
        call = q2.q4_linear_grouped if c["fmt"] == "q4" else q2.q2_linear_grouped
        return call(state["x"], state["offsets"], *state["w"], row_index=state["index"], bias=state["bias"],
                    activation=c["act"], gated=c["gated"], out_dtype=DTYPES[c["out"]])
    if op == "route":
        return tuple(q2.q2_route(state["logits"], c["top"], renormalize=c["renorm"]))
    return q2.q2_combine(state["z"], state["slot"], state["weight"], residual=state["residual"],
                         out_dtype=DTYPES[c["out"]])


# ---------------------------------------------------------------------------
# the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _weights64(w, fmt):
    """Weights from a table of every byte's codes."""
    bits, codes = (2, 4) if fmt == "q2" else (4, 2)
    table = torch.tensor([[byte >> (bits * i) & (2 ** bits - 1) for i in range(codes)] for byte in range(256)],
                         dtype=torch.float64, device=DEV)
    q = table[w[0].int()].flatten(-2)
    spread = [t.double().repeat_interleave(BLOCK, dim=-1) for t in w[1:]]
    return q.sub_(spread[1] if fmt == "q4" else 1.0).mul_(spread[0])


def _act64(name, v):
    if name == "none":
        return v
    if name == "relu":
        return torch.maximum(v, torch.zeros_like(v))
    if name == "silu":
        return v * torch.special.expit(v)
    if name == "gelu":
        return v * torch.special.ndtr(v)
    u = math.sqrt(8 / math.pi) * (v + 0.044715 * v ** 3)      # (1 + tanh(u / 2)) / 2 is the logistic function of u
    return v * torch.special.expit(u)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("fused", "grouped"):
        gated, act = case["gated"], case["act"]

        def finish(z):
            if not gated:
                return _act64(act, z)
            a, b = z.chunk(2, dim=-1)
            return _act64(act, a) * b

        if case["op"] == "fused":
            x = s["x"].double()
            z = torch.matmul(x, _weights64(s["w"], case["fmt"]).mT)
            if case["rank"]:
                z += x.matmul(s["A"].double().mT).matmul(s["B"].double().mT)
            if case["bias"]:
                z += s["bias"].double()
            y = finish(z)
            if case["gate"]:
                y = y * s["gate"].double()
            return y + s["residual"].double() if case["residual"] else y
        out, at = [], s["offsets"].tolist()
        for e in range(case["experts"]):
            rows = torch.arange(at[e], at[e + 1], device=DEV)
            x = s["x"][rows if s["index"] is None else s["index"].long()[rows]].double()
            z = torch.matmul(x, _weights64([t[e] for t in s["w"]], case["fmt"]).mT)
            out.append(finish(z + s["bias"][e].double() if case["bias"] else z))
        return torch.cat(out)
    if case["op"] == "route":
        v = s["logits"].double()
        t, e, top = case["tokens"], case["experts"], case["top"]
        # the rank of an expert: how many are larger, or equal with a lower number
        lower = torch.ones((e, e), dtype=torch.bool, device=DEV).tril(-1)
        expert = torch.full((t, top), -1, device=DEV)
        for lo in range(0, t, 1024):
            a, b = v[lo:lo + 1024, :, None], v[lo:lo + 1024, None, :]
            rank = ((b > a) | ((b == a) & lower)).sum(2)
            rank[v[lo:lo + 1024] == -math.inf] = e
            tok, ex = (rank < top).nonzero(as_tuple=True)
            expert[lo + tok, rank[tok, ex]] = ex
        live = expert >= 0
        chosen = torch.where(live, v.gather(1, expert.clamp(min=0)), -math.inf)
        whole = (chosen if case["renorm"] else v).logsumexp(1, keepdim=True)
        weight = torch.where(live, (chosen - whole).exp(), 0.0)
        flat = expert.flatten()
        count = torch.stack([(flat == n).sum() for n in range(e)])
        offsets = torch.cat([count.new_zeros(1), count.cumsum(0)])
        slot, token = torch.full_like(flat, -1), torch.full_like(flat, -1)
        for n in range(e):
            at = (flat == n).nonzero().squeeze(1)
            slot[at] = offsets[n] + torch.arange(at.numel(), device=DEV)
            token[offsets[n]:offsets[n + 1]] = at // top
        return expert.int(), weight, offsets.int(), token.int(), slot.view(t, top).int()
    y = torch.zeros((case["tokens"], case["n"]), dtype=torch.float64, device=DEV)
    for j in range(case["top"]):
        live = s["slot"][:, j] >= 0
        y[live] += s["z"][s["slot"][live, j].long()].double() * s["weight"][live, j, None].double()
    return y + s["residual"].double() if case["residual"] else y
