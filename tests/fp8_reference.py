"""The 8-bit product and the expert layer in 64 bits, and what the kernels may be off by.

An e4m3 x e4m3 or bf16 x e4m3 product is exact in fp32.  A sum of fp32 numbers, in any order, by additions that are off
by at most one unit in the last place (2^-23 of the partial sum, which is never above the sum of magnitudes) is off by
at most 2^-23 of the sum of magnitudes for each addition on an element's way: at most 128 within a block, one for each
block after that (whatever the split, some more for its parts), and SLACK for scales and joins.
"""
from __future__ import annotations

import torch

DEV = "cuda"
BLOCK = 128
ULP = 2.0 ** -23
HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2
HALF_F32 = 2.0 ** -24
SLACK = 32
# Below fp32's normal numbers there is less than full precision, or none: whatever is that small may be off by this.
TINY = 2.0 ** -126


def blocks(n):
    return -(-n // BLOCK)


def sum_ulps(k):
    """Additions on the way of one product to its sum of k, in blocks of 128."""
    return BLOCK + blocks(k) + SLACK


def quantise(x, block_rows):
    """(codes as float8, scales) of a bf16 matrix, in fp32 as the definition says (on x's device)."""
    r, c = x.shape
    s = torch.empty(-(-r // block_rows), blocks(c), device=x.device)
    y = torch.empty(r, c, device=x.device)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            at = (slice(i * block_rows, (i + 1) * block_rows), slice(j * BLOCK, (j + 1) * BLOCK))
            top = x[at].float().abs().amax()  # NaN if any is
            s[i, j] = torch.maximum(top / torch.full_like(top, 448), torch.full_like(top, 2.0 ** -126))  # by a number it is a product
            y[at] = x[at].float() / s[i, j]
    return y.clamp(-448, 448).to(torch.float8_e4m3fn), s


def spread(s, rows, cols, block_rows=BLOCK):
    """A scale for every element, in 64 bits."""
    return s.double().repeat_interleave(block_rows, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :cols]


def values(codes, s, block_rows=BLOCK):
    return codes.double() if s is None else codes.double() * spread(s, *codes.shape, block_rows)


def codes_of(gen, rows, cols, block_rows, spare=0):
    """Random codes of every magnitude (a view with padded rows) and positive scales."""
    width = -(-cols // 16) * 16 + spare
    x = torch.randn(rows, width, generator=gen, device=DEV) * 60
    c = x.clamp(-448, 448).to(torch.float8_e4m3fn)[:, :cols]
    s = torch.exp(torch.randn(-(-rows // block_rows), blocks(cols), generator=gen, device=DEV)) * 0.01
    return c, s


def product(x, xs, w, ws, out_dtype):
    """(the product in 64 bits, what each element may be off by)."""
    a, b = values(x, xs, 1), values(w, ws)
    y = a @ b.T
    tol = sum_ulps(x.shape[1]) * ULP * (a.abs() @ b.abs().T)
    return y, tol + (HALF_BF16 * (y.abs() + tol) if out_dtype == torch.bfloat16 else 0)


def assert_within(got, want, tol, what):
    got = got.double()
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= tol)
    if bool(bad.any()):
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {i}: {got[i].item()} for "
                             f"{want[i].item()} (+- {tol[i].item():.3g})")


# ------------------------------------------------------------------------------------ expert layers

def experts(g, gen, E, H, I, Is=0, e4m3=True, bias=False, gate=True, spread_logits=1.5):
    """A handle of random weights."""
    def matrices(*shape):
        w = torch.randn(*shape, generator=gen, device=DEV) * shape[-1] ** -0.5
        if not e4m3:
            return w.bfloat16(), None
        s = torch.exp(0.3 * torch.randn(*shape[:-2], blocks(shape[-2]), blocks(shape[-1]), generator=gen, device=DEV)) * 0.01
        full = s.repeat_interleave(BLOCK, -2)[..., :shape[-2], :].repeat_interleave(BLOCK, -1)[..., :shape[-1]]
        return (w / full).clamp(-448, 448).to(torch.float8_e4m3fn), s
    gu, gus = matrices(E, 2, I, H)
    dn, dns = matrices(E, H, I)
    kw = {}
    if Is:
        kw["shared_gate_up"], kw["shared_gate_up_scale"] = matrices(2, Is, H)
        kw["shared_down"], kw["shared_down_scale"] = matrices(H, Is)
        if gate:
            kw["shared_gate"] = (torch.randn(H, generator=gen, device=DEV) * H ** -0.5).bfloat16()
    router = (spread_logits * torch.randn(E, H, generator=gen, device=DEV) * H ** -0.5).bfloat16()
    rb = 0.1 * torch.randn(E, generator=gen, device=DEV) if bias else None
    return g.Experts(gu, dn, gus, dns, router=router, router_bias=rb, **kw)


def scores(x, ex, scoring):
    """(logits, scores, what the choice goes by, what a logit may be off by), in 64 bits."""
    a, r = x.double(), ex.router.double()
    logits = a @ r.T
    off = (a.abs() @ r.abs().T) * (x.shape[1] / 32 + SLACK) * ULP
    s = torch.sigmoid(logits) if scoring == "sigmoid" else torch.softmax(logits, -1)
    by = logits if ex.router_bias is None else s + ex.router_bias.double()
    return logits, s, by, off


def assert_choice(ids, weights, x, ex, top_k, scoring, renormalise, scale):
    """The ids are a top_k choice, largest first, within what scores may be off by; the weights go with them."""
    logits, s, by, off = scores(x, ex, scoring)
    ids = ids.long()
    assert bool(((ids >= 0) & (ids < s.shape[1])).all())
    assert all(len(set(r)) == top_k for r in ids.tolist())
    # a score moves by at most what the logits move by (sigmoid: a quarter of it; softmax: twice it, relative)
    room = 4 * off.amax(1, keepdim=True) + 8 * ULP * (1 + by.abs().amax(1, keepdim=True))
    got = by.gather(1, ids)
    want = by.sort(dim=1, descending=True, stable=True)
    assert bool(((got - want.values[:, :top_k]).abs() <= room).all()), "not the largest scores in order"
    gap = want.values[:, :-1] - want.values[:, 1:]
    clear = (torch.nn.functional.pad(gap, (0, 1), value=1.0)[:, :top_k] > room) | (torch.nn.functional.pad(gap, (0, 1), value=1.0)[:, :top_k] == 0)
    clear = clear & torch.nn.functional.pad(clear, (1, 0), value=True)[:, :top_k]
    assert bool((ids == want.indices[:, :top_k])[clear].all()), "ties go to the lowest index"
    w = s.gather(1, ids)
    if renormalise:
        w = w / w.sum(1, keepdim=True)
    w = w * scale
    assert_within(weights, w, w.abs() * (4 * off.amax(1, keepdim=True) + 64 * ULP) + (1 + abs(scale)) * TINY, "weights")


def layer(x, ex, ids, weights, weight_off=0.0):
    """(the layer's rows for this routing in 64 bits, what each may be off by).  weight_off: relative, of the weights and the
    shared expert's gate."""
    T, H = x.shape
    a = x.double()
    y, mag, tol = (torch.zeros(T, H, dtype=torch.float64, device=x.device) for _ in range(3))

    def add(rows, f, gu, gus, dn, dns):
        gate, up, down = (values(m, s) for m, s in ((gu[0], None if gus is None else gus[0]),
                                                    (gu[1], None if gus is None else gus[1]), (dn, dns)))
        xa = a[rows]
        g, u = xa @ gate.T, xa @ up.T
        dg, du = ((xa.abs() @ m.abs().T) * sum_ulps(H) * ULP for m in (gate, up))
        silu = g * torch.sigmoid(g)
        h = silu * u
        # silu's slope is at most 1.1; the hidden value keeps 16 bits: off by 2^-16 of itself; 16 ulps for the arithmetic
        dh = 1.1 * dg * u.abs() + silu.abs() * du + 1.1 * dg * du + (2.0 ** -16 + 16 * ULP) * h.abs() + TINY
        one = h @ down.T
        size = h.abs() @ down.abs().T
        off = dh @ down.abs().T + sum_ulps(down.shape[1]) * ULP * size
        y[rows] += f[:, None] * one
        mag[rows] += f.abs()[:, None] * one.abs()
        tol[rows] += f.abs()[:, None] * (off + weight_off * one.abs())

    for e in sorted(set(ids.flatten().tolist())):
        if 0 <= e < ex.gate_up.shape[0]:
            f = (weights.double() * (ids == e)).sum(1)
            rows = (ids == e).any(1).nonzero()[:, 0]
            add(rows, f[rows], ex.gate_up[e], None if ex.gate_up_scale is None else ex.gate_up_scale[e], ex.down[e],
                None if ex.down_scale is None else ex.down_scale[e])
    if ex.shared_gate_up is not None:
        f = torch.ones(T, dtype=torch.float64, device=x.device)
        if ex.shared_gate is not None:
            f = torch.sigmoid(a @ ex.shared_gate.double())
        add(torch.arange(T, device=x.device), f, ex.shared_gate_up, ex.shared_gate_up_scale, ex.shared_down,
            ex.shared_down_scale)
    tol = tol + (ids.shape[1] + 4) * ULP * mag + TINY
    return y, tol + HALF_BF16 * (y.abs() + tol)


def assert_layer(out, x, ex, ids, weights, what="layer"):
    """weights are the ones that the call used (its own, or the given ones), so they count as exact; the shared gate's
    sigmoid moves by at most what its logit does."""
    off = 0.0
    if ex.shared_gate is not None:
        off = float((x.double().abs() @ ex.shared_gate.double().abs()).amax()) * (x.shape[1] / 32 + SLACK) * ULP + 16 * ULP
    want, tol = layer(x, ex, ids, weights, off)
    assert_within(out, want, tol, what)
