"""Quantising to e4m3 by blocks, and the 8-bit product, against their definitions."""
from __future__ import annotations

import math

import pytest
import torch

from tests.fp8_reference import DEV, assert_within, blocks, codes_of, product, quantise, values
from tests.gpu_common import Guarded, lib
from tests.test_gpu_fresh_thread import on_a_fresh_thread

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def gen_of(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def same_codes(got, want):
    """Equal bytes; any NaN for NaN."""
    a, b = got.contiguous().view(torch.uint8), want.contiguous().view(torch.uint8)
    return bool(((a == b) | (((a & 0x7F) == 0x7F) & ((b & 0x7F) == 0x7F))).all())


def same_floats(got, want):
    return bool(((got == want) | (got.isnan() & want.isnan())).all())


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols,stride", [(1, 1, 1), (1, 128, 128), (3, 5, 5), (130, 129, 129), (64, 2048, 2048),
                                              (257, 1000, 1016), (128, 300, 333), (5, 16384, 16384), (300, 127, 128)])
def test_quantize_is_the_definition(rows, cols, stride, block_rows):
    g = lib()
    gen = gen_of(rows * 7 + cols)
    x = torch.randn(rows, stride, generator=gen, device=DEV) * torch.exp(2 * torch.randn(rows, 1, generator=gen, device=DEV))
    x = x.bfloat16()[:, :cols]
    wide = -(-cols // 16) * 16 + 32
    room = Guarded((rows, wide), torch.uint8)
    room.t.fill_(0xAB)
    sc = Guarded((-(-rows // block_rows), blocks(cols)), torch.float32)
    codes, scales = g.gdn_fp8_quantize(x, block_rows, room.t.view(E4M3)[:, :cols], sc.t)
    want, ws = quantise(x, block_rows)
    assert torch.equal(scales, ws) and same_codes(codes, want)
    assert bool((room.t[:, cols:] == 0xAB).all())
    room.check("codes"), sc.check("scales")
    c2, s2 = g.gdn_fp8_quantize(x, block_rows)
    assert same_codes(c2, want) and torch.equal(s2, ws) and c2.stride(0) % 16 == 0


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_special_values(block_rows):
    """Zeros, the smallest and largest bf16, infinities and NaN, each in a block of its own."""
    g = lib()
    x = torch.zeros(130, 9 * 128 - 3, device=DEV)
    x[:, 128:256] = 2.0 ** -133
    x[:, 256:384] = -3.3895e38
    x[3, 384 + 5] = math.inf
    x[:, 400] = 2.0
    x[2, 512 + 7] = math.nan
    x[:, 520] = 2.0
    x[:, 640:768] = -0.0
    x[:, 768] = -448.0
    x[:, 769:780] = torch.arange(11, device=DEV) * 17.0 - 4.0
    x[:, 896] = 2.0 ** -126 * 448
    x[:, 897] = 2.0 ** -126
    x[:, 1024:] = torch.linspace(-1e-3, 1e-3, x.shape[1] - 1024, device=DEV)
    x = x.bfloat16()
    codes, scales = g.gdn_fp8_quantize(x, block_rows)
    want, ws = quantise(x, block_rows)
    assert same_floats(scales, ws) and same_codes(codes, want)


def test_quantize_many_rows():
    """More rows than a grid's second dimension holds, and offsets beyond 2^31 elements."""
    g = lib()
    x = torch.randn(140000, 16, generator=gen_of(1), device=DEV).bfloat16()
    codes, scales = g.gdn_fp8_quantize(x)
    top = x.float().abs().amax(1, keepdim=True)
    s = (top / torch.full_like(top, 448)).clamp(min=2.0 ** -126)
    assert torch.equal(scales, s) and same_codes(codes, (x.float() / s).to(E4M3))
    big = torch.empty(3, 1 << 30, dtype=torch.bfloat16, device=DEV)[:, :200]
    big.copy_(torch.randn(3, 200, generator=gen_of(2), device=DEV))
    codes, scales = g.gdn_fp8_quantize(big)
    want, ws = quantise(big, 1)
    assert torch.equal(scales, ws) and same_codes(codes, want)


SHAPES = [(1, 1, 1), (1, 128, 128), (2, 7, 15), (1, 5000, 2048), (3, 200, 16), (16, 128, 4000), (17, 384, 256),
          (31, 1000, 1000), (64, 2048, 640), (65, 129, 127), (100, 640, 2041), (128, 128, 128), (129, 257, 384),
          (200, 96, 5120), (256, 1024, 512), (300, 1000, 130), (777, 515, 257), (1024, 2048, 512), (1500, 300, 1290)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,N,K", SHAPES)
def test_product(T, N, K, dtype):
    g = lib()
    gen = gen_of(T + 3 * N + 5 * K)
    x, xs = codes_of(gen, T, K, 1)
    w, ws = codes_of(gen, N, K, 128, spare=16)
    out = Guarded((T, N), dtype)
    got = g.gdn_fp8_matmul(x, xs, w, ws, out=out.t)
    g.gdn_check_device_errors()
    out.check("out")
    want, tol = product(x, xs, w, ws, dtype)
    assert_within(got, want, tol, f"{T} x {N} x {K}")
    assert torch.equal(got, g.gdn_fp8_matmul(x, xs, w, ws, out_dtype=dtype)), "two calls, the same bits"


# either side of where tiles of 64 rows share their k among 4, 2 or 1 CTAs, and of where tiles of 256 rows begin and share
# theirs, on a device with 152 SMs; many tiles for each CTA; odd everything
BORDERS = [(128, 38 * 64, 640), (100, 39 * 64, 640), (128, 76 * 64, 300), (120, 76 * 64 + 1, 300), (128, 152 * 64, 129),
           (256, 76 * 64, 200), (129, 76 * 64 + 1, 200), (200, 5003, 129), (1500, 1603, 257), (2500, 4099, 1023),
           (70, 9793, 4097), (300, 4096, 4096), (128, 19456, 4000), (128, 19457, 4224)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,N,K", BORDERS)
def test_product_where_tiles_change(T, N, K, dtype):
    test_product(T, N, K, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [1, 3, 8, 250])
@pytest.mark.parametrize("T,N,K", [(5, 129, 256), (130, 384, 200), (513, 250, 128)])
def test_product_into_strided_rows(T, N, K, pad, dtype):
    """Rows of every alignment; what lies between them stays."""
    g = lib()
    gen = gen_of(11)
    x, xs = codes_of(gen, T, K, 1, spare=48)
    w, ws = codes_of(gen, N, K, 128)
    room = torch.full((T, N + pad), 7.25, dtype=dtype, device=DEV)
    g.gdn_fp8_matmul(x, xs, w, ws, out=room[:, :N])
    want, tol = product(x, xs, w, ws, dtype)
    assert_within(room[:, :N], want, tol, "strided")
    assert bool((room[:, N:] == 7.25).all())


@pytest.mark.parametrize("T,N,K", [(5, 200, 300), (200, 400, 300), (1100, 600, 300)])
def test_values_that_are_not_finite_stay_in_their_rows_and_columns(T, N, K):
    g = lib()
    gen = gen_of(12)
    x, xs = codes_of(gen, T, K, 1)
    w, ws = codes_of(gen, N, K, 128)
    clean = g.gdn_fp8_matmul(x, xs, w, ws, out_dtype=torch.float32)
    xs, ws = xs.clone(), ws.clone()
    x[3, 299] = math.nan
    xs[1, 2], xs[2, 0] = math.nan, math.inf
    w[130, 0] = math.nan
    got = g.gdn_fp8_matmul(x, xs, w, ws, out_dtype=torch.float32)
    bad = torch.zeros(T, N, dtype=torch.bool, device=DEV)
    bad[[1, 3]] = True
    bad[2] = True
    bad[:, 130] = True
    assert not bool(got[bad].isfinite().any()) and torch.equal(got[~bad], clean[~bad])
    ws[1, 1] = math.inf  # rows 128 .. 255 of w
    got = g.gdn_fp8_matmul(x, xs, w, ws, out_dtype=torch.float32)
    bad[:, 128:256] = True
    assert not bool(got[bad].isfinite().any()) and torch.equal(got[~bad], clean[~bad])


def test_product_of_extreme_scales():
    """Scales from 2^-126 to 2^100, blocks of zeros, sums that cancel."""
    g = lib()
    gen = gen_of(13)
    T, N, K = 70, 140, 640
    x, _ = codes_of(gen, T, K, 1)
    w, _ = codes_of(gen, N, K, 128)
    x[:, 128:256] = 0
    xs = torch.tensor([2.0 ** -60, 2.0 ** -126, 1.0, 2.0 ** -60, 2.0 ** 40], device=DEV).repeat(T, 1)
    ws = torch.tensor([2.0 ** 60, 2.0 ** 100, 0.5, -2.0 ** 60, 2.0 ** -40], device=DEV).repeat(2, 1)
    for dtype in (torch.bfloat16, torch.float32):
        got = g.gdn_fp8_matmul(x, xs, w, ws, out_dtype=dtype)
        want, tol = product(x, xs, w, ws, dtype)
        assert_within(got, want, tol, "scales")


def test_far_offsets():
    """Codes, weights and results beyond 2^31 elements."""
    g = lib()
    gen = gen_of(14)
    T, N, K = 33000, 66000, 64
    x, xs = codes_of(gen, T, K, 1)
    w, ws = codes_of(gen, N, K, 128)
    got = g.gdn_fp8_matmul(x, xs, w, ws)
    for lo in (0, 16000, T - 100):
        want, tol = product(x[lo:lo + 100], xs[lo:lo + 100], w, ws, torch.bfloat16)
        assert_within(got[lo:lo + 100], want, tol, f"rows from {lo}")
    del got
    wide = torch.zeros(40, 1 << 27, dtype=torch.uint8, device=DEV).view(E4M3)[:, :K]  # 5 GiB apart at the far end
    wide.view(torch.uint8).copy_(w[:40].contiguous().view(torch.uint8))
    a = g.gdn_fp8_matmul(x[:50], xs[:50], wide, ws[:1])
    b = g.gdn_fp8_matmul(wide, xs[:40], w[:50], ws[:1])
    want, tol = product(x[:50], xs[:50], w[:40], ws[:1], torch.bfloat16)
    assert_within(a, want, tol, "far weights")
    want, tol = product(w[:40], xs[:40], w[:50], ws[:1], torch.bfloat16)
    assert_within(b, want, tol, "far rows")


def test_quantised_product_together():
    """Activations and weights quantised and multiplied: within what two roundings to e4m3 cost."""
    g = lib()
    gen = gen_of(15)
    T, N, K = 150, 300, 1000
    x, w = (torch.randn(r, K, generator=gen, device=DEV).bfloat16() for r in (T, N))
    (xc, xs), (wc, ws) = g.gdn_fp8_quantize(x), g.gdn_fp8_quantize(w, 128)
    got = g.gdn_fp8_matmul(xc, xs, wc, ws, out_dtype=torch.float32)
    want, tol = product(xc, xs, wc, ws, torch.float32)
    assert_within(got, want, tol, "product")
    # a value is off by 2^-4 of itself, or half the least step 2^-9 of its scale
    a, b = x.double(), w.double()
    da = a.abs() * 2.0 ** -4 + 2.0 ** -10 * xs.double().repeat_interleave(128, 1)[:, :K]
    db = b.abs() * 2.0 ** -4 + 2.0 ** -10 * ws.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    assert bool(((values(xc, xs, 1) - a).abs() <= da * (1 + 1e-6)).all())
    off = da @ b.abs().T + a.abs() @ db.T + da @ db.T
    assert_within(got, a @ b.T, off + tol, "against bf16")


def test_no_rows():
    g = lib()
    x, xs = torch.empty(0, 256, device=DEV, dtype=E4M3), torch.empty(0, 2, device=DEV)
    w, ws = codes_of(gen_of(16), 30, 256, 128)
    assert g.gdn_fp8_matmul(x, xs, w, ws).shape == (0, 30)
    assert g.gdn_fp8_matmul(w, torch.ones(30, 2, device=DEV), x, xs).shape == (30, 0)
    c, s = g.gdn_fp8_quantize(torch.empty(0, 100, device=DEV, dtype=torch.bfloat16))
    assert c.shape == (0, 100) and s.shape == (0, 1)


@pytest.mark.parametrize("T,N,K", [(1, 1024, 2048), (200, 512, 640), (1300, 640, 512)])
def test_graph_side_stream_and_fresh_thread(T, N, K):
    """Captured with the quantisation before it and replayed on new values; on another stream; as a thread's first call."""
    g = lib()
    gen = gen_of(17)
    x = torch.randn(T, K, generator=gen, device=DEV).bfloat16()
    w, ws = codes_of(gen, N, K, 128)
    out = torch.empty(T, N, dtype=torch.bfloat16, device=DEV)
    codes, scales = g.gdn_fp8_quantize(x)
    first = g.gdn_fp8_matmul(codes, scales, w, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c2, s2 = g.gdn_fp8_quantize(x)
        assert torch.equal(first, g.gdn_fp8_matmul(c2, s2, w, ws))
    given = g.gdn_fp8_matmul(codes, scales, w, ws, stream=side)
    side.synchronize()
    assert torch.equal(first, given)
    torch.cuda.synchronize()
    on_a_fresh_thread(lambda: g.gdn_fp8_matmul(codes, scales, w, ws, out=out, stream=torch.cuda.default_stream()))
    torch.cuda.synchronize()
    assert torch.equal(first, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gdn_fp8_quantize(x, codes=codes, scales=scales)
        g.gdn_fp8_matmul(codes, scales, w, ws, out=out)
    for seed in (1, 2):
        x.copy_(torch.randn(T, K, generator=gen_of(seed), device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        want, tol = product(codes, scales, w, ws, torch.bfloat16)
        assert_within(out, want, tol, "replayed")
        assert same_codes(codes, quantise(x[:3], 1)[0] if T < 3 else g.gdn_fp8_quantize(x)[0])
    g.gdn_check_device_errors()


def test_refusals():
    g = lib()
    x, xs = codes_of(gen_of(18), 4, 100, 1)
    w, ws = codes_of(gen_of(18), 30, 100, 128)
    for bad in (lambda: g.gdn_fp8_matmul(x, xs[:, :0], w, ws), lambda: g.gdn_fp8_matmul(x[:, :99], xs, w, ws),
                lambda: g.gdn_fp8_matmul(x, xs, w, ws, out=torch.empty(30, 4, device=DEV)),
                lambda: g.gdn_fp8_matmul(x.t(), xs, w, ws), lambda: g.gdn_fp8_quantize(xs.bfloat16(), block_rows=2)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: g.gdn_fp8_matmul(x.float(), xs, w, ws), lambda: g.gdn_fp8_matmul(x, xs.double(), w, ws),
                lambda: g.gdn_fp8_matmul(x, xs, w, ws, out_dtype=torch.float16), lambda: g.gdn_fp8_quantize(xs)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(g.GdnError) as e:  # rows of 100 bytes
        g.gdn_fp8_matmul(x.contiguous(), xs, w, ws)
    assert e.value.name == "GDN_ERR_MISALIGNED"


@pytest.mark.parametrize("T", [1, 17])
def test_product_of_the_longest_rows(T):
    """k = 2^31 - 1: nearly all codes are 0, the others stand at the ends and in the middle."""
    g = lib()
    K, N = 2 ** 31 - 1, 2
    at = torch.tensor([0, 1, 127, 128, 2 ** 30 + 5, K - 129, K - 128, K - 17, K - 16, K - 15, K - 2, K - 1], device=DEV)
    gen = gen_of(19)

    def matrix(rows):
        c = torch.zeros(rows, K + 1, dtype=torch.uint8, device=DEV)
        few = torch.randn(rows, at.numel(), generator=gen, device=DEV).to(E4M3)
        c[:, at] = few.view(torch.uint8)
        c[:, K] = 0x7E  # behind the end: not read
        return c.view(E4M3)[:, :K], few.double()
    (x, xf), (w, wf) = matrix(T), matrix(N)
    out = g.gdn_fp8_matmul(x, torch.ones(T, blocks(K), device=DEV), w, torch.ones(1, blocks(K), device=DEV),
                           out_dtype=torch.float32)
    g.gdn_check_device_errors()
    # zeros add nothing: a product is in at most as many sums as there are products, and the joins
    assert_within(out, xf @ wf.T, (at.numel() + 16) * 2.0 ** -23 * (xf.abs() @ wf.abs().T), "long rows")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,N,K", [(5, 200, 300), (16, 200, 300), (60, 400, 300), (200, 400, 300), (1100, 600, 300)])
def test_nan_gives_nan_and_infinite_scales_what_is_not_finite(T, N, K, dtype):
    g = lib()
    gen = gen_of(20)
    x, xs = codes_of(gen, T, K, 1)
    w, ws = codes_of(gen, N, K, 128)
    clean = g.gdn_fp8_matmul(x, xs, w, ws, out_dtype=dtype)
    x[0, 7], w[3, 299], xs[1, 2], ws[1, 0] = math.nan, math.nan, math.nan, math.nan
    xs[2, 0] = math.inf
    nan, room = (torch.zeros(T, N, dtype=torch.bool, device=DEV) for _ in range(2))
    nan[:2], nan[:, 3], nan[:, 128:256] = True, True, True
    room[2] = True
    room &= ~nan
    got = g.gdn_fp8_matmul(x, xs, w, ws, out_dtype=dtype)
    assert bool(got[nan].isnan().all()) and not bool(got[room].isfinite().any())
    assert bool(got[room].isinf().any()) and torch.equal(got[~nan & ~room], clean[~nan & ~room])
    ws = ws.clone()
    ws[0, 1] = -math.inf
    got = g.gdn_fp8_matmul(x, xs, w, ws, out_dtype=dtype)
    room[:, :128] = True
    room &= ~nan
    assert bool(got[nan].isnan().all()) and not bool(got[room].isfinite().any())
    assert torch.equal(got[~nan & ~room], clean[~nan & ~room])
