"""The operators of a softmax-attention layer over a paged key/value cache, as a serving program calls them.

Four operators: ``prepare`` (per-head RMS norm and position rotation of q and k, k and v written to
the pages, bf16 or 8 bits), ``read`` (the pages back to dense rows), ``chunk`` (attention of new
tokens over the cache) and ``token`` (the same for one token of each sequence).
"""
import math

import torch

own = False

EPS = 1e-6
SPARE_PAGES = 3


# ------------------------------------------------------------------------------------ cases

def listed():
    hybrid = {"hq": 16, "hkv": 2, "dim": 256, "rot": 64}    # a hybrid's attention layer: wide heads, a quarter rotated
    square = {"hq": 32, "hkv": 8, "dim": 128, "rot": 128}   # a common dense layer: the whole head rotated
    triple = {"hq": 48, "hkv": 16, "dim": 128, "rot": 128}  # this library's own 48 / 16 heads: three queries to a key head
    return [
        # one decode step's new tokens, 64 sequences, 8-bit cache: a call that is all latency
        {"name": "prepare_step_64", "op": "prepare", **hybrid, "cache": "e4m3", "page": 64, "half": True,
         "seqs": 64, "q_lo": 1, "q_hi": 1, "past_lo": 100, "past_hi": 20000},
        # a long prompt's tokens, 16-bit cache, rotation of neighbouring pairs
        {"name": "prepare_prompt_8192", "op": "prepare", **square, "cache": "bf16", "page": 16, "half": False,
         "seqs": 1, "q_lo": 8192, "q_hi": 8192, "past_lo": 0, "past_hi": 0},
        # a mixed batch of chunks of every length, far positions, 8-bit cache
        {"name": "prepare_ragged_e4m3", "op": "prepare", **hybrid, "cache": "e4m3", "page": 64, "half": True,
         "seqs": 24, "q_lo": 1, "q_hi": 4111, "past_lo": 0, "past_hi": 200000},
        # a stored prefix handed to another program: one long sequence out of an 8-bit cache
        {"name": "read_prefix_32k_e4m3", "op": "read", **hybrid, "cache": "e4m3", "page": 64,
         "seqs": 1, "q_lo": 32768, "q_hi": 32768, "past_lo": 0, "past_hi": 0},
        # many short sequences' rows, small pages, from the middle of each
        {"name": "read_ragged_bf16", "op": "read", **square, "cache": "bf16", "page": 16,
         "seqs": 33, "q_lo": 5, "q_hi": 900, "past_lo": 0, "past_hi": 100},
        # a whole prompt at once
        {"name": "chunk_prompt_8192", "op": "chunk", **square, "cache": "bf16", "page": 16, "gate": False,
         "seqs": 1, "q_lo": 8192, "q_hi": 8192, "past_lo": 0, "past_hi": 0},
        # one scheduling step of a long prompt: 2048 new tokens behind 30 thousand, gated output
        {"name": "chunk_2048_after_30k", "op": "chunk", **hybrid, "cache": "bf16", "page": 64, "gate": True,
         "seqs": 1, "q_lo": 2048, "q_hi": 2048, "past_lo": 30001, "past_hi": 30001},
        # chunks of several prompts together, 8-bit cache
        {"name": "chunk_ragged_e4m3", "op": "chunk", **hybrid, "cache": "e4m3", "page": 64, "gate": True,
         "seqs": 8, "q_lo": 17, "q_hi": 1500, "past_lo": 300, "past_hi": 9000},
        # a short follow-up question: few rows, a small cache, three queries to a key head
        {"name": "chunk_17_after_1000", "op": "chunk", **triple, "cache": "bf16", "page": 16, "gate": False,
         "seqs": 1, "q_lo": 17, "q_hi": 17, "past_lo": 1000, "past_hi": 1000},
        # one user's next token: the latency of a single call
        {"name": "token_1_at_4000", "op": "token", **hybrid, "cache": "bf16", "page": 64, "gate": True,
         "seqs": 1, "q_lo": 1, "q_hi": 1, "past_lo": 4000, "past_hi": 4000},
        # a server's step: sequences of every length
        {"name": "token_64_ragged", "op": "token", **hybrid, "cache": "bf16", "page": 64, "gate": True,
         "seqs": 64, "q_lo": 1, "q_hi": 1, "past_lo": 30, "past_hi": 30000},
        # a large batch on the 8-bit cache
        {"name": "token_256_e4m3", "op": "token", **square, "cache": "e4m3", "page": 16, "gate": False,
         "seqs": 256, "q_lo": 1, "q_hi": 1, "past_lo": 500, "past_hi": 8000},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["prepare", "read", "chunk", "token"])
    dim = rng.choice([128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    case = {"op": op, "dim": dim, "hkv": hkv, "hq": hkv * rng.choice([1, 2, 3, 4, 6, 8]),
            "rot": rng.choice([32, 64, 96, 128]), "cache": rng.choice(["bf16", "e4m3"]),
            "page": rng.choice([16, 32, 64, 128]), "seqs": log(1, 100)}
    if op == "token":
        q = past = 0
        case.update(gate=rng.random() < 0.5, q_lo=1, q_hi=1, past_lo=log(1, 200), past_hi=log(200, 16000))
        case["past_hi"] = min(case["past_hi"], 400000 // case["seqs"] + 200)
    elif op == "chunk":
        case.update(gate=rng.random() < 0.5, q_lo=log(1, 40), q_hi=log(40, 2000), past_lo=rng.choice([0, log(1, 500)]),
                    past_hi=log(500, 12000))
        case["seqs"] = min(case["seqs"], 12, max(1, 6000 // case["q_hi"]))
    elif op == "prepare":
        case.update(half=rng.random() < 0.5, q_lo=log(1, 40), q_hi=log(40, 8000), past_lo=0, past_hi=log(1, 100000))
        case["q_hi"] = case["q_hi"] * 16 // max(16, case["hq"]) + 40
        case["seqs"] = min(case["seqs"], max(1, 24000 * 16 // max(16, case["hq"]) // case["q_hi"]))
        case["past_hi"] = min(case["past_hi"], 1500000 // case["seqs"])
    else:
        case.update(q_lo=log(1, 40), q_hi=log(40, 30000), past_lo=0, past_hi=log(1, 2000))
        case["seqs"] = min(case["seqs"], max(1, 30000 // case["q_hi"]))
    return case


def _spread(lo, hi, n, shift):
    """n lengths between lo and hi, evenly over their logarithm, in a fixed order that is not sorted."""
    if n == 1:
        return [hi]
    at = [round(math.exp(math.log(lo + 1) + (math.log(hi + 1) - math.log(lo + 1)) * i / (n - 1))) - 1 for i in range(n)]
    step = next(s for s in (7, 11, 13, 17, 19, 23, 29) if math.gcd(s, n) == 1)
    return [at[(i * step + shift) % n] for i in range(n)]


def _lengths(case):
    """New tokens and cached tokens (the new ones among them) of each sequence."""
    q = [max(1, x) for x in _spread(case["q_lo"], case["q_hi"], case["seqs"], 0)]
    past = _spread(case["past_lo"], case["past_hi"], case["seqs"], 5)
    return q, [a + b for a, b in zip(q, past)]


def work(case):
    q, kv = _lengths(case)
    T, hq, hkv, D = sum(q), case["hq"], case["hkv"], case["dim"]
    row = 2 * hkv * (2 * D if case["cache"] == "bf16" else D + 1)  # one cached position, keys and values
    if case["op"] == "prepare":
        return {"bytes": T * (2 * (hq + 2 * hkv) * D + 2 * hq * D + row), "flops": T * (hq + hkv) * D * 8}
    if case["op"] == "read":
        return {"bytes": T * (row + 4 * hkv * D), "flops": 0}
    gate = 2 * T * hq * D if case["gate"] else 0
    seen = sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(q, kv))
    return {"bytes": sum(kv) * row + 4 * T * hq * D + gate, "flops": 4 * D * hq * seen}


# ------------------------------------------------------------------------------------ inputs

def _two(e):
    """2^e exactly, as 32-bit floats, for whole e of the normal range."""
    return ((e + 127).to(torch.int32) << 23).view(torch.float32)


def _quantise(x):
    """8-bit codes of rows x and the exponent byte of each row's power of two."""
    a = x.float().abs().amax(-1)
    m, e = torch.frexp(a)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(a > 0, e, -117).clamp(min=-117)
    codes = (x.float() * _two(-e)[..., None]).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    hq, hkv, D, page, bits8 = case["hq"], case["hkv"], case["dim"], case["page"], case["cache"] == "e4m3"
    q_lens, kv_lens = _lengths(case)
    T, N = sum(q_lens), len(q_lens)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    need = [-(-x // page) for x in kv_lens]
    s = {"op": case["op"], "max_q": max(q_lens), "max_kv": max(kv_lens), "total": T, "bits8": bits8, "gate": None,
         "dims": (hq, hkv, D, page), "half": case.get("half"), "one": case["op"] == "token" or max(q_lens) == 1,
         "scale": 1.0 / math.sqrt(D)}
    s["cu"] = torch.tensor([0] + q_lens, dtype=torch.int32).cumsum(0, dtype=torch.int32).cuda()
    s["kv_lens"] = torch.tensor(kv_lens, dtype=torch.int32).cuda()
    past = [b - a for a, b in zip(q_lens, kv_lens)]
    s["starts"] = torch.tensor(past, dtype=torch.int32).cuda()

    # the pages of the sequences, scattered over the pool as a server that has run for a while has them; a write
    # needs the new tokens' pages alone, the others are one page that it never touches
    wide, first = max(need), [(x // page if case["op"] == "prepare" else 0) for x in past]
    pool = sum(n - f for n, f in zip(need, first)) + SPARE_PAGES
    order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32).cpu().tolist()
    table, at = torch.full((N, wide), order[-1], dtype=torch.int32), 0
    for n in range(N):
        table[n, first[n]:need[n]] = torch.tensor(order[at:at + need[n] - first[n]], dtype=torch.int32)
        at += need[n] - first[n]
    s["table"] = table.cuda()
    s["k_scale"] = s["v_scale"] = None
    if case["op"] == "prepare":
        kind = torch.float8_e4m3fn if bits8 else torch.bfloat16
        s["k"], s["v"] = (torch.zeros(pool, hkv, page, D, dtype=kind, device="cuda") for _ in range(2))
        if bits8:
            s["k_scale"], s["v_scale"] = (torch.full((pool, hkv, page), 127, dtype=torch.uint8, device="cuda") for _ in range(2))
    else:
        s["k"], s["v"] = normal(pool, hkv, page, D) * 1.3, normal(pool, hkv, page, D)
        if bits8:
            s["k"], s["k_scale"] = _quantise(s["k"])
            s["v"], s["v_scale"] = _quantise(s["v"])

    if case["op"] == "prepare":
        # one projection's output: queries, keys and values of a token side by side
        s["qkv"] = normal(T, (hq + 2 * hkv) * D) * 2
        s["q_w"], s["k_w"] = 1 + 0.1 * normal(D), 1 + 0.1 * normal(D)
        # positions scaled for long contexts: an eightfold longer range than the base was made for
        s["freqs"] = 1e6 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"]) / 8
        s["m"] = 1.1
        s["q_out"] = torch.empty(T, hq, D, dtype=torch.bfloat16, device="cuda")
    elif case["op"] == "read":
        s["k_out"], s["v_out"] = (torch.empty(T, hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    else:
        s["q"] = normal(T, hq, D) * 1.3
        s["gate"] = normal(T, hq, D) if case["gate"] else None
        s["out"] = torch.empty(T, hq, D, dtype=torch.bfloat16, device="cuda")
    return s


# ------------------------------------------------------------------------------------ one pass

def run(s):
    if own:
        return _own(s)
    return {"prepare": _prepare, "read": _read, "chunk": _attention, "token": _attention}[s["op"]](s)


def _own(s):
    import linear_attention_ssm_gb300 as gdn
    hq, hkv, D, page = s["dims"]
    cache = gdn.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    if s["op"] == "prepare":
        q, k, v = s["qkv"].view(s["total"], hq + 2 * hkv, D).split([hq, hkv, hkv], dim=1)
        gdn.gdn_attn_prepare(q, k, v, cache, s["table"], s["kv_lens"], cu_seqlens=None if s["one"] else s["cu"],
                             q_norm_w=s["q_w"], k_norm_w=s["k_w"], rope_freqs=s["freqs"], rope_interleaved=not s["half"],
                             rope_scale=s["m"], rms_eps=EPS, q_out=s["q_out"])
        return _written(s, s["q_out"])
    if s["op"] == "read":
        gdn.gdn_attn_cache_read(cache, s["table"], s["cu"], s["k_out"], s["v_out"], starts=s["starts"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if s["op"] == "token":
        return gdn.gdn_attn_decode_step(s["q"], cache, s["table"], s["kv_lens"], s["scale"], z=s["gate"], out=s["out"])
    return gdn.gdn_attn_prefill(s["q"], cache, s["table"], s["kv_lens"], s["cu"], s["scale"], z=s["gate"], out=s["out"])


def _written(s, q):
    out = {"q": q, "k": s["k"], "v": s["v"]}
    if s["bits8"]:
        out.update(k_scale=s["k_scale"].view(torch.float8_e8m0fnu), v_scale=s["v_scale"].view(torch.float8_e8m0fnu))
    return out


def _places(s, starts):
    """Sequence, position, page and row in the page of every token."""
    t = torch.arange(s["total"], device="cuda")
    seq = torch.searchsorted(s["cu"][1:], t, right=True)
    pos = starts[seq] + t - s["cu"][seq]
    return seq, pos, s["table"][seq, pos // s["dims"][3]], pos % s["dims"][3]


def _norm_rotate(x, w, pos, s):
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    angle = pos.double()[:, None] * s["freqs"]
    c, n = (torch.cos(angle) * s["m"]).float()[:, None], (torch.sin(angle) * s["m"]).float()[:, None]
    r = 2 * s["freqs"].numel()
    if s["half"]:
        a, b = y[..., :r // 2], y[..., r // 2:r]
        turned = torch.cat([a * c - b * n, b * c + a * n], -1)
    else:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    return torch.cat([turned, y[..., r:]], -1).bfloat16()


def _prepare(s):
    hq, hkv, D, page = s["dims"]
    q, k, v = s["qkv"].view(s["total"], hq + 2 * hkv, D).split([hq, hkv, hkv], dim=1)
    _, pos, at, row = _places(s, s["starts"])
    q, k = _norm_rotate(q, s["q_w"], pos, s), _norm_rotate(k, s["k_w"], pos, s)
    if s["bits8"]:
        (k, ks), (v, vs) = _quantise(k), _quantise(v)
        s["k_scale"][at, :, row] = ks
        s["v_scale"][at, :, row] = vs
        s["k"].view(torch.uint8)[at, :, row] = k.view(torch.uint8)
        s["v"].view(torch.uint8)[at, :, row] = v.view(torch.uint8)
    else:
        s["k"][at, :, row] = k
        s["v"][at, :, row] = v
    return _written(s, q)


def _value(codes, scale):
    return codes.float() if scale is None else codes.float() * _two(scale.int() - 127)[..., None]


def _read(s):
    _, _, at, row = _places(s, s["starts"])
    if s["bits8"]:
        k, v = (s[x].view(torch.uint8)[at, :, row].view(torch.float8_e4m3fn) for x in ("k", "v"))
        return {"k": _value(k, s["k_scale"][at, :, row]).bfloat16(), "v": _value(v, s["v_scale"][at, :, row]).bfloat16()}
    return {"k": s["k"][at, :, row], "v": s["v"][at, :, row]}


def _attention(s):
    """Every sequence padded to the longest one, scores in 32 bits."""
    hq, hkv, D, page = s["dims"]
    N, Q, P = s["kv_lens"].numel(), s["max_q"], -(-s["max_kv"] // page)
    pages = s["table"][:, :P].long()

    def gathered(x, scale):
        x = x.view(torch.uint8)[pages].view(x.dtype) if scale is not None else x[pages]
        x = _value(x, None if scale is None else scale[pages])
        return x.permute(0, 2, 1, 3, 4).reshape(N, hkv, P * page, D)

    k, v = gathered(s["k"], s["k_scale"]), gathered(s["v"], s["v_scale"])
    i, lens = torch.arange(Q, device="cuda"), s["cu"].diff()
    token = (s["cu"][:-1, None] + i).clamp(max=s["total"] - 1)
    q = s["q"].float()[token].view(N, Q, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4).reshape(N, hkv, -1, D)
    scores = (q @ k.transpose(-1, -2)).mul_(s["scale"]).view(N, hkv, hq // hkv, Q, P * page)
    pos = s["starts"][:, None] + i
    hidden = torch.arange(P * page, device="cuda") > pos[..., None]
    scores.masked_fill_(hidden[:, None, None], float("-inf"))
    scores.sub_(scores.amax(-1, keepdim=True)).exp_()
    total = scores.sum(-1, keepdim=True)
    o = (scores.view(N, hkv, -1, P * page) @ v).view(N, hkv, hq // hkv, Q, D) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(N, Q, hq, D)[i < lens[:, None]]
    if s["gate"] is not None:
        o = o * torch.sigmoid(s["gate"].float())
    return o.bfloat16()


# ------------------------------------------------------------------------------------ the definition, in 64 bits

def _power(e):
    """2^e exactly, as 64-bit floats."""
    return ((e + 1023) << 52).view(torch.float64)


def exact(case, seed):
    s = prepare(case, seed)
    hq, hkv, D, page = s["dims"]
    cu, kv_lens, group = s["cu"].tolist(), s["kv_lens"].tolist(), hq // hkv
    starts = [kv - (cu[n + 1] - cu[n]) for n, kv in enumerate(kv_lens)]

    def cached(x, scale, n, lo, hi):
        """Rows lo .. hi - 1 of sequence n as [heads, rows, D] doubles."""
        first = lo // page
        ids = s["table"][n, first:-(-hi // page)].long()
        y = x.view(torch.uint8)[ids].view(x.dtype).double() if scale is not None else x[ids].double()
        if scale is not None:
            y = y * _power(scale[ids].long() - 127)[..., None]
        return y.transpose(0, 1).reshape(hkv, -1, D)[:, lo - first * page:hi - first * page]

    if case["op"] == "read":
        def rows(x, scale):
            return torch.cat([cached(x, scale, n, st, kv).transpose(0, 1) for n, (st, kv) in enumerate(zip(starts, kv_lens))])
        return {"k": rows(s["k"], s["k_scale"]), "v": rows(s["v"], s["v_scale"])}

    if case["op"] == "prepare":
        heads = s["qkv"].double().view(-1, hq + 2 * hkv, D)
        pos = torch.cat([torch.arange(st, kv, device="cuda", dtype=torch.float64) for st, kv in zip(starts, kv_lens)])
        r = case["rot"]
        z = torch.polar(torch.full_like(pos, s["m"])[:, None].expand(-1, r // 2), pos[:, None] * s["freqs"][None])[:, None]

        def turned(x, w):
            y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * w.double()
            first = torch.arange(r // 2, device="cuda") * (1 if case["half"] else 2)
            second = first + (r // 2 if case["half"] else 1)
            c = torch.complex(y[..., first], y[..., second]) * z
            y[..., first], y[..., second] = c.real, c.imag
            return y

        q, k, v = turned(heads[:, :hq], s["q_w"]), turned(heads[:, hq:hq + hkv], s["k_w"]), heads[:, hq + hkv:]
        out = {"q": q}
        for name, x in (("k", k), ("v", v)):
            pages = s[name].double()
            scales = torch.ones(pages.shape[:3], dtype=torch.float64, device="cuda")
            if s["bits8"]:
                top = x.abs().amax(-1, keepdim=True)
                top = top.bfloat16().double()
                two = _power(torch.ceil(torch.log2(top / 448.0) - 1e-6).long())  # top has 8 bits: no ratio above a power of two is as near to it
                x = x / two
            for n, (st, kv) in enumerate(zip(starts, kv_lens)):
                at = torch.arange(st, kv, device="cuda")
                ids = s["table"][n].long()[at // page]
                pages[ids, :, at % page] = x[cu[n]:cu[n + 1]]
                if s["bits8"]:
                    scales[ids, :, at % page] = two[cu[n]:cu[n + 1], :, 0]
            out[name] = pages
            if s["bits8"]:
                out[name + "_scale"] = scales
        return out

    out = torch.empty(s["total"], hq, D, dtype=torch.float64, device="cuda")
    for n, (st, kv) in enumerate(zip(starts, kv_lens)):
        k, v = (cached(s[x], s[x + "_scale"], n, 0, kv) for x in ("k", "v"))
        for lo in range(cu[n], cu[n + 1], 256):
            hi = min(lo + 256, cu[n + 1])
            q = s["q"][lo:hi].double().view(-1, hkv, group, D).permute(1, 2, 0, 3)
            a = torch.einsum("hgtd,hjd->hgtj", q, k) * s["scale"]
            pos = st + torch.arange(lo - cu[n], hi - cu[n], device="cuda")
            a = a.masked_fill(torch.arange(kv, device="cuda")[None] > pos[:, None], -math.inf)
            out[lo:hi] = torch.einsum("hgtj,hjd->thgd", torch.softmax(a, -1), v).reshape(hi - lo, hq, D)
    if s["gate"] is not None:
        out = out / (1 + torch.exp(-s["gate"].double()))
    return out
