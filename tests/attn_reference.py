"""The paged-cache attention layer's operators in 64 bits, sequence by sequence, and the error each
result may have (roundings counted from the formulas the kernels state)."""
from __future__ import annotations

import math

import torch

DEV = "cuda"


def two(e):
    """2^e exactly for whole e (the GPU's pow is not)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def quantise(x):
    """Rows x (float64 of bf16 values) -> (codes as float64, exponent bytes): the largest finite
    magnitude a, the least e >= -117 with a <= 448 * 2^e, x / 2^e rounded to e4m3 by numpy-like rules."""
    a = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).abs().amax(-1)
    e = torch.full_like(a, -117)
    for k in range(-117, 128):
        e = torch.where((a > 448 * 2.0 ** (k - 1)) & (k > -117), torch.full_like(a, float(k)), e)
    y = x / two(e)[..., None]
    # e4m3: three fraction bits, steps of 2^-9 below 2^-6, ties to even
    size = torch.where(torch.isfinite(y), y.abs(), torch.ones_like(y)).clamp(min=2.0 ** -6)
    step = two(torch.frexp(size)[1] - 1 - 3)
    codes = torch.round(y / step) * step
    return torch.where(torch.isfinite(y), codes, torch.full_like(y, math.nan)), (e + 127).to(torch.uint8)


def positions(q_lens, kv_lens):
    """(sequence, position) of every packed row."""
    seq = [n for n, q in enumerate(q_lens) for _ in range(q)]
    pos = [kv - q + i for q, kv in zip(q_lens, kv_lens) for i in range(q)]
    return seq, pos


def norm_rotate(x, w, pos, freqs, interleaved, magnitude, eps):
    """(y, the magnitude its rounding errors go by) of rows x [T, H, D] at positions pos [T]."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    size = y.abs()
    if freqs is None:
        return y, size
    R = 2 * freqs.numel()
    j = torch.arange(R // 2, device=x.device)
    a_at, b_at = (2 * j, 2 * j + 1) if interleaved else (j, j + R // 2)
    theta = torch.tensor(pos, dtype=torch.float64, device=x.device)[:, None] * freqs
    c, s = magnitude * theta.cos()[:, None], magnitude * theta.sin()[:, None]
    a, b = y[..., a_at], y[..., b_at]
    out, big = y.clone(), size.clone()
    out[..., a_at], out[..., b_at] = a * c - b * s, b * c + a * s
    big[..., a_at] = big[..., b_at] = magnitude * (a.abs() + b.abs())
    return out, big


def dense_rows(cache, table_row, hi):
    """Rows 0 .. hi - 1 of one sequence: k, v as float64 [Hkv, hi, D]."""
    page = cache.k.shape[2]
    ids = table_row[:-(-hi // page)].long()

    def rows(x, scale):
        y = x.view(torch.uint8)[ids].view(x.dtype).double() if scale is not None else x[ids].double()
        if scale is not None:
            y = y * two(scale[ids].long() - 127)[..., None]
        return y.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])[:, :hi]
    return rows(cache.k, cache.k_scale), rows(cache.v, cache.v_scale)


def attention(q, cache, table, q_lens, kv_lens, scale, z=None):
    """(out, the error it may have), float64 [T, Hq, D].

    Counted: scores are fp32 sums of D products (D * 2^-24 of the sum of magnitudes, and 2^-22 of
    the score's own size for its scaling and subtraction), so each weight is off by at most that
    relatively; the weights are rounded to bf16 (2^-8); numerator and denominator both carry the error;
    sums over n keys add n * 2^-24; the result is rounded to bf16 (2^-8).  e4m3: the queries are
    rounded to binary16 after division by a power of two that leaves the largest below 2 (2^-25 of it
    where they leave the normal range), the weights, times 2^7, to binary16: 2^-11, or 2^-25 of 2^-7 of a unit
    that is at most twice the largest value, for each key; a key or value row far below the largest
    may lose 2^-32 of that."""
    hq, D = q.shape[1], q.shape[2]
    out, tol = [torch.zeros(q.shape, dtype=torch.float64, device=q.device) for _ in range(2)]
    e4m3 = cache.k_scale is not None
    first = 0
    for n, (ql, kv) in enumerate(zip(q_lens, kv_lens)):
        lo, first = first, first + ql
        if ql == 0 or kv == 0:
            continue
        k, v = dense_rows(cache, table[n], kv)
        g = hq // k.shape[0]
        qd = q[lo:lo + ql].double().view(ql, -1, g, D).permute(1, 2, 0, 3)
        s = torch.einsum("hgtd,hjd->hgtj", qd, k) * scale
        mag = torch.einsum("hgtd,hjd->hgtj", qd.abs(), k.abs()) * scale
        pos = torch.arange(kv - ql, kv, device=q.device)
        hidden = torch.arange(kv, device=q.device)[None] > pos[:, None]
        s = s.masked_fill(hidden, -math.inf)
        top = s.amax(-1, keepdim=True).clamp(min=-1e300)
        w = torch.exp(s - top)
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total.clamp(min=1e-300), torch.zeros_like(w))
        rel = (D * 2.0 ** -24 * mag + 2.0 ** -22 * (s.abs() + top.abs())).masked_fill(hidden, 0.0).amax(-1, keepdim=True)
        o = torch.einsum("hgtj,hjd->hgtd", w, v)
        size = torch.einsum("hgtj,hjd->hgtd", w, v.abs())
        if e4m3:
            rel = rel + 2.0 ** -32 * scale * k.abs().max() * qd.abs().sum(-1, keepdim=True)
            rel = rel + 2.0 ** -25 * scale * (qd.abs().amax(-1)[..., None] * k.abs().sum(-1)[:, None, None]).amax(-1, keepdim=True)
        err = (2.0 ** (-11 if e4m3 else -8) + 2 * rel + 2 * kv * 2.0 ** -24 + 2.0 ** -20) * size
        if e4m3:
            err = err + kv * 2.0 ** -31 * v.abs().amax((1, 2))[:, None, None, None]
        pack = lambda x: x.permute(2, 0, 1, 3).reshape(ql, hq, D)  # noqa: E731
        o, err = pack(o), pack(err)
        if z is not None:
            gate = torch.sigmoid(z[lo:lo + ql].double())
            o, err = o * gate, err * gate + o.abs() * 2.0 ** -20
        out[lo:lo + ql], tol[lo:lo + ql] = o, err + 2.0 ** -8 * (o.abs() + err)
    return out, tol


def assert_within(got, want, tol, what):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN in other places"
    over = (got - want).abs() - tol
    worst = torch.nan_to_num(over, nan=-1.0).max().item() if over.numel() else -1.0
    assert worst <= 0, f"{what}: an element is {worst:.3g} further off than its rounding errors allow"
