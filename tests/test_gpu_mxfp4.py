"""MXFP4 quantisation and product on the GPU against their definitions in
binary64.

Quantisation is exact up to the element's one rounding, which binary64
reproduces, so codes, scales and read-back values are compared bit for bit.
The product sums exact products in float32: with n = k terms the error of any
summation order is below n 2^-24 sum |a w|, plus the tensor core's truncation
of aligned addends (a few 2^-23 of the largest per instruction), for which the
bound below takes 2^-20 of sum |a w| at k <= 4096, then one rounding to the
output type (unit roundoff 2^-8, 2^-11 or 2^-24 of the value)."""
import math

import pytest
import torch

import diffusion_transformer_mlp_gb300 as fc2
import _mx as mx

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
HALF_ULP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


def rnd(shape, seed, dtype=torch.float32, spread=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    if spread:
        x = x * torch.exp2(torch.randn(shape, generator=g, device="cuda") * spread)
    return x.to(dtype)


def check_bytes(t, x):
    rows, cols = x.shape
    code, e = mx.encode(mx.pad_cols(x.double()))
    got = mx.unpack(t.qdata.reshape(-1, code.shape[1] // 2)[:rows])
    assert torch.equal(got, code)
    assert torch.equal(mx.tile_scales(t.scales, rows, cols), e)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 32), (3, 33), (2, 127), (130, 257), (5, 1344), (1, 5376), (33, 512),
                                       (300, 2001), (257, 96)])
def test_quantize_bytes(rows, cols, dtype):
    x = rnd((rows, cols), rows * 7 + cols, dtype, spread=3.0)
    t = fc2.mxfp4_quantize(x)
    check_bytes(t, x)
    back = fc2.mxfp4_dequantize(t, torch.float32)
    assert torch.equal(back.double(), mx.values(x))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 0), (0, 3), (8, 8), (3, 5)])
def test_quantize_strided_and_misaligned(dtype, offset, pad):
    rows, cols = 37, 416
    buf = rnd((rows * (cols + pad) + offset,), 5, dtype)
    x = buf[offset:].view(rows, cols + pad)[:, :cols]
    t = fc2.mxfp4_quantize(x)
    check_bytes(t, x)
    out = torch.full((rows * (cols + pad) + offset + 8,), 7.0, dtype=dtype, device="cuda")
    view = out[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    fc2.mxfp4_dequantize(t, out=view)
    assert torch.equal(view.double(), mx.values(x))
    rest = torch.ones_like(out, dtype=torch.bool)
    rest[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = False
    assert bool((out[rest] == 7.0).all())


def test_quantize_midpoints_signs_and_extremes():
    """Every midpoint of the grid and its neighbours under several scales, signed
    zeros, the largest and the smallest numbers."""
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, 0.0, 6.0], device="cuda")
    near = torch.cat([mids, mids * (1 + 2.0 ** -23), mids * (1 - 2.0 ** -23)])
    block = torch.cat([near, torch.tensor([-0.0, 4.0], device="cuda")])
    rows = [block * s * 2.0 ** e for s in (1.0, -1.0) for e in (-126, -100, -10, 0, 1, 60, 124)]
    big = torch.full((32,), 3.4028234663852886e38, device="cuda")
    tiny = torch.full((32,), 2.0 ** -149, device="cuda")
    mixed = torch.where(torch.arange(32, device="cuda") % 2 == 0, big, -tiny)
    sub = torch.arange(32, device="cuda").float() * 2.0 ** -130
    x = torch.stack(rows + [big, -big, tiny, mixed, sub, torch.zeros(32, device="cuda"),
                            -torch.zeros(32, device="cuda")])
    t = fc2.mxfp4_quantize(x)
    check_bytes(t, x)
    assert torch.equal(fc2.mxfp4_dequantize(t, torch.float32).double(), mx.values(x))


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_nonfinite_blocks(dtype):
    x = rnd((4, 200), 9, dtype)
    x[0, 5] = math.nan
    x[1, 40] = math.inf
    x[2, 199] = -math.inf
    t = fc2.mxfp4_quantize(x)
    check_bytes(t, x)
    back = fc2.mxfp4_dequantize(t, dtype)
    want = torch.zeros(4, 200, dtype=torch.bool, device="cuda")
    want[0, :32] = want[1, 32:64] = want[2, 192:] = True
    assert torch.equal(torch.isnan(back), want)
    assert torch.equal(back[~want].double(), mx.values(x)[~want].to(dtype).double())


@pytest.mark.parametrize("dtype", DTYPES)
def test_dequantize_every_code_and_scale(dtype):
    """All 256 scale codes times all 16 element codes: exact in bfloat16 and
    float32, one rounding in float16."""
    t = fc2.empty_mxfp4(256, 32)
    t.qdata.zero_()
    t.qdata[:, :16] = (torch.arange(16, device="cuda") * 16 + (15 - torch.arange(16, device="cuda"))).to(torch.uint8)
    s = torch.zeros(2, 1, 32, 4, 4, dtype=torch.uint8, device="cuda")
    s.permute(0, 3, 2, 1, 4).reshape(256, 4)
    e = torch.arange(256, device="cuda", dtype=torch.uint8).reshape(2, 4, 32)
    s[:, 0, :, :, 0] = e.transpose(1, 2)
    t.scales.copy_(s.flatten())
    got = fc2.mxfp4_dequantize(t, dtype)
    want = mx.decode(mx.unpack(t.qdata)[:, :32], torch.arange(256, device="cuda", dtype=torch.uint8).unsqueeze(1))
    if dtype is torch.float16:
        want = want.float().to(dtype).double()  # float32 holds every value
    elif dtype is torch.bfloat16:
        want = want.float().to(dtype).double()
        assert torch.equal(want.float().double()[:255], want[:255])
    else:
        want = want.float().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(got.double()[ok], want[ok])


def product_ref(x, w):
    a, b = mx.values(x), mx.values(w)
    return a @ b.T, a.abs() @ b.abs().T


def check_product(out, ref, mag, dtype):
    bound = HALF_ULP[dtype] * 1.01 * ref.abs() + 2.0 ** -20 * mag + (2.0 ** -25 if dtype is torch.float16 else 0.0)
    err = (out.double() - ref).abs()
    worst = float((err / bound.clamp(min=1e-300)).max())
    assert worst <= 1.0, worst


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 128, 128), (1, 1000, 4096), (3, 129, 257), (16, 256, 1344),
                                   (17, 300, 511), (32, 127, 2000), (61, 640, 1024), (64, 1, 640), (65, 513, 384),
                                   (128, 256, 256), (129, 1000, 769), (300, 2049, 1152), (513, 384, 4096),
                                   (1000, 777, 129)])
def test_gemm(m, n, k, dtype):
    x, w = rnd((m, k), m + k, torch.float32), rnd((n, k), n * 3 + k, torch.float32)
    x = torch.where(torch.rand_like(x) < 0.01, x * 20, x)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = fc2.mxfp4_gemm(fc2.mxfp4_quantize(x), fc2.mxfp4_quantize(w), dtype=dtype, status=status)
    ref, mag = product_ref(x, w)
    assert out.shape == (m, n) and out.dtype is dtype and int(status) == 0
    check_product(out, ref, mag, dtype)


@pytest.mark.parametrize("m,n,k", [(2, 200, 512), (50, 130, 300), (200, 260, 512), (700, 1100, 640)])
def test_gemm_exact_when_sums_are_exact(m, n, k):
    """Small whole numbers: every partial sum is exact in float32, so the output
    is the exact product rounded once, whatever the order of the sum."""
    g = torch.Generator(device="cuda").manual_seed(m)
    x = torch.tensor([0.0, 1, 2, 3, 4, 6], device="cuda")[torch.randint(0, 6, (m, k), generator=g, device="cuda")]
    w = torch.tensor([0.0, 1, -2, 3, -4, 6], device="cuda")[torch.randint(0, 6, (n, k), generator=g, device="cuda")]
    a, b = fc2.mxfp4_quantize(x), fc2.mxfp4_quantize(w)
    ref = mx.values(x) @ mx.values(w).T
    for dtype in DTYPES:
        assert torch.equal(fc2.mxfp4_gemm(a, b, dtype=dtype), ref.to(dtype))


@pytest.mark.parametrize("m,n", [(5, 333), (200, 400), (600, 391), (300, 392), (257, 520)])
def test_gemm_output_view_leaves_the_rest(m, n):
    k = 320
    x, w = rnd((m, k), 1), rnd((n, k), 2)
    a, b = fc2.mxfp4_quantize(x), fc2.mxfp4_quantize(w)
    want = fc2.mxfp4_gemm(a, b)
    for off, pad in ((0, 9), (1, 0), (8, 16), (16, 7)):
        buf = torch.full((m * (n + pad) + off + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
        view = buf[off:off + m * (n + pad)].view(m, n + pad)[:, :n]
        fc2.mxfp4_gemm(a, b, out=view)
        assert torch.equal(view, want)
        rest = torch.ones_like(buf, dtype=torch.bool)
        rest[off:off + m * (n + pad)].view(m, n + pad)[:, :n] = False
        assert bool((buf[rest] == 3.0).all())


@pytest.mark.parametrize("m", [4, 100, 500])
def test_gemm_nan_blocks_stay_in_their_rows(m):
    n, k = 300, 512
    x, w = rnd((m, k), 3), rnd((n, k), 4)
    want = fc2.mxfp4_gemm(fc2.mxfp4_quantize(x), fc2.mxfp4_quantize(w))
    x[2, 100], w[17, 300] = math.nan, math.inf
    got = fc2.mxfp4_gemm(fc2.mxfp4_quantize(x), fc2.mxfp4_quantize(w))
    nan = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    nan[2], nan[:, 17] = True, True
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("m", [3, 200])
def test_gemm_ignores_bytes_past_the_rows(m):
    """Scale bytes of rows past the operands (same 128-row tile) may hold anything."""
    n, k = 200, 384
    a, b = fc2.mxfp4_quantize(rnd((m, k), 5)), fc2.mxfp4_quantize(rnd((n, k), 6))
    outs = []
    for fill in (0, 255):
        for t, rows in ((a, m), (b, n)):
            s = t.scales.view(-1, 3, 32, 4, 4).permute(0, 3, 2, 1, 4)
            s.reshape(-1, 12)  # shape check only: the loop writes through the permuted view
            r = torch.arange(s.shape[0] * 128, device="cuda").view(s.shape[0], 4, 32)
            s[r >= rows] = fill
        outs.append(fc2.mxfp4_gemm(a, b))
    assert torch.equal(outs[0], outs[1]) and bool(torch.isfinite(outs[0]).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,n,k", [(1, 300, 5376), (7, 129, 1000), (16, 256, 512), (40, 500, 333), (300, 260, 1030)])
def test_linear_is_quantize_then_gemm(m, n, k, dtype):
    x = rnd((m, k + 5), m, dtype)[:, 2:k + 2]
    w = fc2.mxfp4_quantize(rnd((n, k), n))
    out = fc2.mxfp4_linear(x, w)
    assert out.dtype is dtype
    ref, mag = product_ref(x, fc2.mxfp4_dequantize(w, torch.float32))
    check_product(out, ref, mag, dtype)
    assert torch.equal(out, fc2.mxfp4_linear(x.contiguous(), w))


def test_linear_reproducible_on_another_stream():
    x, w = rnd((9, 2048), 1, torch.bfloat16), fc2.mxfp4_quantize(rnd((1000, 2048), 2))
    want = fc2.mxfp4_linear(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = [fc2.mxfp4_linear(x, w) for _ in range(20)]
    s.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_linear_in_a_graph():
    x, w = rnd((4, 1024), 1, torch.bfloat16), fc2.mxfp4_quantize(rnd((256, 1024), 2))
    out = fc2.mxfp4_linear(x, w)
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = fc2.mxfp4_linear(x, w)
    out.zero_()
    g.replay()
    assert torch.equal(out, want)


def test_linear_without_rows():
    w = fc2.mxfp4_quantize(rnd((64, 128), 1))
    assert fc2.mxfp4_linear(torch.empty(0, 128, device="cuda"), w).shape == (0, 64)


def test_refusals():
    x = rnd((4, 64), 1, torch.bfloat16)
    w = fc2.mxfp4_quantize(rnd((8, 64), 2))
    with pytest.raises(ValueError):
        fc2.mxfp4_quantize(x.double())
    with pytest.raises(ValueError):
        fc2.mxfp4_quantize(x.t())
    with pytest.raises(ValueError):
        fc2.mxfp4_quantize(x.cpu())
    with pytest.raises(ValueError):
        fc2.mxfp4_linear(x[:, :32], w)
    with pytest.raises(ValueError):
        fc2.mxfp4_linear(x, w, out=torch.empty(4, 9, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        fc2.mxfp4_gemm(fc2.MXFP4Tensor(w.qdata[:1].contiguous(), w.scales, 8, 64), w)
    with pytest.raises(ValueError):
        fc2.mxfp4_dequantize(w, torch.int32)
    with pytest.raises(fc2.NVFP4Error):
        fc2.mxfp4_quantize(x[:1].expand(4, 64))
