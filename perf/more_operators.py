"""8-bit products and expert layers around the sublayers, as a serving program calls them.

Three operators: ``quantise`` (bf16 values to e4m3 codes with one fp32 scale for 128 values of a row, or for a block
of 128 x 128), ``product`` (activations times weights in that form) and ``experts`` (a whole mixture-of-experts layer
for a few tokens: router, choice, gated experts, weighted sum).
"""
import math

import torch

own = False

BLOCK = 128
TOP = 448.0            # the largest e4m3 value
LEAST = 2.0 ** -126    # of a scale


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step's rows before a projection: all latency
        {"name": "quantise_step_64", "op": "quantise", "rows": 64, "cols": 2048, "block_rows": 1},
        # a long prompt's gated-norm output (48 heads of 128) before the output projection
        {"name": "quantise_prompt_16384", "op": "quantise", "rows": 16384, "cols": 6144, "block_rows": 1},
        # a checkpoint's bf16 projection of odd sizes brought to 8 bits at load time
        {"name": "quantise_weight_odd", "op": "quantise", "rows": 10001, "cols": 4099, "block_rows": 128},
        # one user's next token through the input projection (10,240 conv channels and 6,144 gate values)
        {"name": "product_token_1", "op": "product", "t": 1, "n": 16384, "k": 2048, "out": "bf16"},
        # a decode step of 64 sequences through the output projection: little weight, a long sum
        {"name": "product_step_64", "op": "product", "t": 64, "n": 2048, "k": 6144, "out": "bf16"},
        # a ragged batch of chunks, no size a multiple of anything, 32-bit results for what follows
        {"name": "product_ragged_777_fp32", "op": "product", "t": 777, "n": 5003, "k": 2041, "out": "fp32"},
        # a scheduling step's chunk through the output projection
        {"name": "product_chunk_2048", "op": "product", "t": 2048, "n": 4096, "k": 6144, "out": "bf16"},
        # a long prompt through the input projection: the largest product
        {"name": "product_prompt_8192", "op": "product", "t": 8192, "n": 16384, "k": 4096, "out": "bf16"},
        # one user's next token through an expert layer, 8-bit weights
        {"name": "experts_token_1", "op": "experts", "t": 1, "e": 64, "k": 8, "h": 2048, "i": 1024, "shared": 0,
         "weights": "e4m3", "score": "softmax", "bias": False},
        # eight sequences' step, sigmoid scores with a bias on the choice, a shared expert behind its own gate
        {"name": "experts_step_8_shared", "op": "experts", "t": 8, "e": 128, "k": 10, "h": 2048, "i": 512,
         "shared": 512, "weights": "e4m3", "score": "sigmoid", "bias": True},
        # the rows of a speculative step, 16-bit weights
        {"name": "experts_verify_17_bf16", "op": "experts", "t": 17, "e": 32, "k": 4, "h": 2048, "i": 1408, "shared": 0,
         "weights": "bf16", "score": "softmax", "bias": False},
        # the largest step: 64 sequences, nearly every one of 288 experts is chosen by some
        {"name": "experts_step_64", "op": "experts", "t": 64, "e": 288, "k": 8, "h": 4096, "i": 1536, "shared": 1536,
         "weights": "e4m3", "score": "sigmoid", "bias": True},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["quantise", "product", "product", "experts"])
    if op == "quantise":
        case = {"op": op, "rows": log(1, 16384), "cols": log(128, 8192), "block_rows": rng.choice([1, 128])}
        case["rows"] = min(case["rows"], 100000000 // case["cols"])
        return case
    if op == "product":
        t, n, k = log(1, 8192), log(64, 16384), log(64, 8192)
        if rng.random() < 0.5:  # most projections are whole blocks
            n, k = -(-n // BLOCK) * BLOCK, -(-k // BLOCK) * BLOCK
        t = min(t, max(1, 8192 * 16384 * 4096 // (n * k)))
        return {"op": op, "t": t, "n": n, "k": k, "out": rng.choice(["bf16", "bf16", "fp32"])}
    e = rng.choice([8, 32, 60, 128, 256])
    h, i = 16 * log(16, 256), 16 * log(8, 128)
    e = min(e, max(8, 5000000000 // (3 * h * i)))
    return {"op": op, "t": log(1, 64), "e": e, "k": rng.choice([1, 2, 4, 6, 8]), "h": h, "i": i,
            "shared": rng.choice([0, 0, i, 16 * log(8, 64)]), "weights": rng.choice(["e4m3", "e4m3", "bf16"]),
            "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5}


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    if case["op"] == "quantise":
        r, c = case["rows"], case["cols"]
        return {"bytes": 3 * r * c + 4 * -(-r // case["block_rows"]) * _blocks(c), "flops": 2 * r * c}
    if case["op"] == "product":
        t, n, k = case["t"], case["n"], case["k"]
        scales = 4 * (t + _blocks(n)) * _blocks(k)
        return {"bytes": (t + n) * k + scales + t * n * (2 if case["out"] == "bf16" else 4), "flops": 2 * t * n * k}
    t, e, k, h, i, s = (case[x] for x in ("t", "e", "k", "h", "i", "shared"))
    chosen = e * (1 - (1 - k / e) ** t)  # different experts, on average
    one = 3 * h * (2 if case["weights"] == "bf16" else 1)
    nbytes = chosen * one * i + one * s + 2 * e * h + 4 * t * h + 8 * t * k + (2 * h if s else 0)
    return {"bytes": int(nbytes), "flops": 6 * t * h * (k * i + s) + 2 * t * e * h}


# ------------------------------------------------------------------------------------ inputs

def _rows16(rows, cols):
    """Room for codes whose rows begin at multiples of 16 bytes."""
    return torch.zeros(rows, -(-cols // 16) * 16, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[:, :cols]


def _quantise(x, block_rows):
    """Codes and scales of x [..., rows, cols]."""
    r, c = x.shape[-2:]
    br, bc = -(-r // block_rows), _blocks(c)
    x = torch.nn.functional.pad(x.float(), (0, bc * BLOCK - c, 0, br * block_rows - r))
    x = x.unflatten(-1, (bc, BLOCK)).unflatten(-3, (br, block_rows))
    top = x.abs().amax((-3, -1))
    scale = (top / torch.full_like(top, TOP)).clamp(min=LEAST)  # a division in earnest: by a number it is a product
    codes = (x / scale[..., :, None, :, None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    return codes.flatten(-2, -1).flatten(-3, -2)[..., :r, :c], scale


def _values(codes, scale, block_rows=BLOCK):
    """The 32-bit values of codes [..., rows, cols] with their scales."""
    r, c = codes.shape[-2:]
    scale = scale.repeat_interleave(block_rows, -2)[..., :r, :].repeat_interleave(BLOCK, -1)[..., :c]
    return codes.float() * scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    s = dict(case)
    if case["op"] == "quantise":
        r, c, b = case["rows"], case["cols"], case["block_rows"]
        # values of very different rows and columns, as a norm's outlier channels make them
        s["x"] = normal(r, c) * torch.exp(normal(r, 1).float()).bfloat16() * torch.exp(normal(1, c).float()).bfloat16()
        s["codes"] = _rows16(r, c)
        s["scales"] = torch.empty(-(-r // b), _blocks(c), dtype=torch.float32, device="cuda")
        return s
    if case["op"] == "product":
        t, n, k = case["t"], case["n"], case["k"]
        s["xc"], s["wc"] = _rows16(t, k), _rows16(n, k)
        codes, s["xs"] = _quantise(normal(t, k) * torch.exp(normal(1, k).float() / 2).bfloat16(), 1)
        s["xc"].copy_(codes)
        codes, s["ws"] = _quantise(normal(n, k) * (k ** -0.5 * torch.exp(normal(n, 1).float() / 4)).bfloat16(), BLOCK)
        s["wc"].copy_(codes)
        s["result"] = torch.empty(t, n, dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32, device="cuda")
        return s
    t, e, k, h, i, sh = (case[x] for x in ("t", "e", "k", "h", "i", "shared"))

    def matrices(count, rows, cols):
        """`count` matrices and their scales (None for 16 bits)."""
        if case["weights"] == "bf16":
            w = torch.empty(count, rows, cols, dtype=torch.bfloat16, device="cuda")
            for j in range(count):
                w[j] = normal(rows, cols) * cols ** -0.5
            return w, None
        w = torch.empty(count, rows, cols, dtype=torch.float8_e4m3fn, device="cuda")
        scale = torch.empty(count, _blocks(rows), _blocks(cols), device="cuda")
        for j in range(count):
            w[j], scale[j] = _quantise(normal(rows, cols) * cols ** -0.5, BLOCK)
        return w, scale

    s["x"] = normal(t, h)
    s["router"] = normal(e, h) * (1.5 * h ** -0.5)
    s["router_bias"] = 0.05 * torch.randn(e, generator=g, device="cuda") if case["bias"] else None
    w, scale = matrices(2 * e, i, h)
    s["gate_up"] = w.view(e, 2, i, h)
    s["gate_up_scale"] = None if scale is None else scale.view(e, 2, _blocks(i), _blocks(h))
    s["down"], s["down_scale"] = matrices(e, h, i)
    for name in ("shared_gate_up", "shared_gate_up_scale", "shared_down", "shared_down_scale", "shared_gate"):
        s[name] = None
    if sh:
        s["shared_gate_up"], s["shared_gate_up_scale"] = matrices(2, sh, h)
        w, scale = matrices(1, h, sh)
        s["shared_down"], s["shared_down_scale"] = w[0], None if scale is None else scale[0]
        s["shared_gate"] = normal(h) * h ** -0.5
    s["result"] = torch.empty(t, h, dtype=torch.bfloat16, device="cuda")
    s["ids"] = torch.empty(t, k, dtype=torch.int32, device="cuda")
    s["chosen_weights"] = torch.empty(t, k, dtype=torch.float32, device="cuda")
    if own:
        import linear_attention_ssm_gb300 as gdn
        s["experts"] = gdn.Experts(
            s["gate_up"], s["down"], s["gate_up_scale"], s["down_scale"], router=s["router"], router_bias=s["router_bias"],
            shared_gate_up=s["shared_gate_up"], shared_down=s["shared_down"],
            shared_gate_up_scale=s["shared_gate_up_scale"], shared_down_scale=s["shared_down_scale"],
            shared_gate=s["shared_gate"])
    return s


ROUTED_SCALE = 1.5  # of the chosen experts' normalised weights


# ------------------------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _own(s)
    return {"quantise": _run_quantise, "product": _run_product, "experts": _run_experts}[s["op"]](s)


def _own(s):
    import linear_attention_ssm_gb300 as gdn
    if s["op"] == "quantise":
        codes, scales = gdn.gdn_fp8_quantize(s["x"], block_rows=s["block_rows"], codes=s["codes"], scales=s["scales"])
        return {"codes": codes, "scales": scales}
    if s["op"] == "product":
        return gdn.gdn_fp8_matmul(s["xc"], s["xs"], s["wc"], s["ws"], out=s["result"])
    out = gdn.gdn_moe_step(s["x"], s["experts"], s["k"], scoring=s["score"], renormalise=True, scale=ROUTED_SCALE,
                           out=s["result"], ids=s["ids"], weights=s["chosen_weights"])
    return {"out": out, "ids": s["ids"], "weights": s["chosen_weights"]}


def _run_quantise(s):
    codes, scales = _quantise(s["x"], s["block_rows"])
    return {"codes": codes, "scales": scales}


def _run_product(s):
    y = _values(s["xc"], s["xs"], 1) @ _values(s["wc"], s["ws"]).T
    return y.to(s["result"].dtype)


def _expert(x, gate_up, gate_up_scale, down, down_scale):
    """The gated expert (or several, one in front of the other) on one row x."""
    if gate_up_scale is not None:
        gate_up, down = _values(gate_up, gate_up_scale), _values(down, down_scale)
    gate_up = gate_up.float() @ x
    gate, up = gate_up[..., 0, :], gate_up[..., 1, :]
    h = gate / (1 + torch.exp(-gate)) * up
    return (down.float() @ h[..., None])[..., 0]


def _run_experts(s):
    x = s["x"].float()
    logits = s["x"].double() @ s["router"].double().T  # 64 bits: the choice is at a border
    score = torch.sigmoid(logits) if s["score"] == "sigmoid" else torch.softmax(logits, -1)
    order = score if s["router_bias"] is None else score + s["router_bias"].double()
    ids = torch.sort(order, dim=-1, descending=True, stable=True).indices[:, :s["k"]]
    w = score.gather(1, ids)
    w = (w / w.sum(-1, keepdim=True) * ROUTED_SCALE).float()
    rows = []
    for t in range(s["t"]):
        at = ids[t]
        scales = (None, None) if s["gate_up_scale"] is None else (s["gate_up_scale"][at], s["down_scale"][at])
        kind = torch.int16 if scales[0] is None else torch.uint8  # rows are moved as whole numbers of their size
        gate_up, down = (s[n].view(kind)[at].view(s[n].dtype) for n in ("gate_up", "down"))
        y = (w[t, :, None] * _expert(x[t], gate_up, scales[0], down, scales[1])).sum(0)
        if s["shared"]:
            open_ = torch.sigmoid((x[t] * s["shared_gate"].float()).sum())
            y = y + open_ * _expert(x[t], s["shared_gate_up"], s["shared_gate_up_scale"], s["shared_down"],
                                    s["shared_down_scale"])
        rows.append(y)
    return {"out": torch.stack(rows).bfloat16(), "ids": ids.int(), "weights": w}


# ------------------------------------------------------------------------------------ the definition, in 64 bits

def _spread(scale, rows, cols, block_rows):
    """A scale for every element: element (i, j) has the scale of block (i // block_rows, j // 128)."""
    i = torch.arange(rows, device="cuda") // block_rows
    j = torch.arange(cols, device="cuda") // BLOCK
    return scale.double()[i][:, j]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantise":
        r, c, b = case["rows"], case["cols"], case["block_rows"]
        x = s["x"].double()
        scale = torch.empty(-(-r // b), _blocks(c), dtype=torch.float64, device="cuda")
        for j in range(_blocks(c)):
            top = x[:, j * BLOCK:(j + 1) * BLOCK].abs().amax(1)
            if b > 1:
                top = torch.stack([part.amax() for part in top.split(b)])
            scale[:, j] = (top / TOP).clamp(min=LEAST)
        return {"codes": x / _spread(scale, r, c, b), "scales": scale}
    if case["op"] == "product":
        t, n, k = case["t"], case["n"], case["k"]
        y = torch.empty(t, n, dtype=torch.float64, device="cuda")
        x = s["xc"].double() * _spread(s["xs"], t, k, 1)
        for lo in range(0, n, 2048):
            hi = min(n, lo + 2048)
            w = s["wc"][lo:hi].double() * _spread(s["ws"][lo // BLOCK:], hi - lo, k, BLOCK)
            y[:, lo:hi] = torch.einsum("tk,nk->tn", x, w)
        return y

    x, k = s["x"].double(), case["k"]
    logits = torch.einsum("th,eh->te", x, s["router"].double())
    if case["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-logits))
    else:
        score = torch.exp(logits - torch.logsumexp(logits, 1, keepdim=True))
    left = score.clone() if s["router_bias"] is None else score + s["router_bias"].double()
    ids = torch.empty(case["t"], k, dtype=torch.int64, device="cuda")
    for j in range(k):  # the largest one of what is left; argmax of the reversed row's last is the lowest index
        best = left.amax(1, keepdim=True)
        ids[:, j] = (left == best).int().argmax(1)
        left.scatter_(1, ids[:, j:j + 1], -math.inf)
    w = torch.gather(score, 1, ids)
    w = ROUTED_SCALE * w / w.sum(1, keepdim=True)
    out = torch.zeros(case["t"], case["h"], dtype=torch.float64, device="cuda")

    def matrix(codes, scale):
        return codes.double() if scale is None else codes.double() * _spread(scale, *codes.shape, BLOCK)

    def add(rows, factor, gate_up, gate_up_scale, down, down_scale):
        scales = (None, None) if gate_up_scale is None else gate_up_scale
        a, b = (torch.einsum("th,ih->ti", x[rows], matrix(gate_up[j], scales[j])) for j in range(2))
        hidden = a * torch.sigmoid(a) * b
        out[rows] += factor[:, None] * torch.einsum("ti,hi->th", hidden, matrix(down, down_scale))

    for e in sorted(set(ids.flatten().tolist())):
        rows, slot = (ids == e).nonzero(as_tuple=True)
        scales = (None, None) if s["gate_up_scale"] is None else (s["gate_up_scale"][e], s["down_scale"][e])
        add(rows, w[rows, slot], s["gate_up"][e], scales[0], s["down"][e], scales[1])
    if case["shared"]:
        every = torch.arange(case["t"], device="cuda")
        add(every, torch.sigmoid(x @ s["shared_gate"].double()), s["shared_gate_up"], s["shared_gate_up_scale"],
            s["shared_down"], s["shared_down_scale"])
    return {"out": out, "ids": ids, "weights": w}
