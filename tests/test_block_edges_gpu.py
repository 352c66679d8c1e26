"""The operators around the layer at the ends of their ranges: rows whose squares leave fp32,
8-bit codes at their borders, scales whose product leaves fp32, and activations far from 0.
Bounds are derived as in test_block_gpu.py: a rounding is off by half a step."""

import math

import pytest
import torch

import diffusion_transformer_moe_b200 as nm
from tests.test_block_gpu import (BF, E4M3, F32, FP8_SHAPES, NORM32, TINY, U, check_linear,
                                  clean, gen, half, norm_ref, product_error, randn, within)

pytestmark = pytest.mark.gpu


def last_step(dtype):
    """Half a step of the type's subnormals."""
    f = torch.finfo(dtype)
    return f.tiny * f.eps / 2


# ---- norm ---------------------------------------------------------------------------------

# a row's size and eps: squares that underflow in part or altogether, that sum just below and
# just above fp32's largest value, or beyond it; eps that is nothing beside them, or as large
ROWS = [(1e-19, 0.0), (1e-20, 0.0), (1e-21, 1e-42), (1e-25, 0.0), (1e-30, 0.0), (1e-37, 0.0),
        (1.0, 0.0), (7e17, 0.0), (8e17, 0.0), (9e17, 0.0), (3e18, 1e37), (1e30, 0.0),
        (1e30, 1e38), (2e37, 0.0)]


def extreme_rows(T, d, dtype, size, seed):
    return randn(gen(seed + d), T, d, dtype=F32, scale=size).to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,d", [(2, 8), (3, 520), (2, 2056), (1, 16384), (1300, 512)])
@pytest.mark.parametrize("size,eps", ROWS)
def test_norm_of_rows_whose_squares_leave_fp32(T, d, dtype, size, eps):
    x = extreme_rows(T, d, dtype, size, 1)
    w = randn(gen(d), d, dtype=dtype)
    n = nm.rms_norm(x, w, eps=eps, out="both")
    clean()
    rstd, y = norm_ref(x, w, float(torch.tensor(eps)))
    within(n.rstd, rstd, rstd * NORM32 + last_step(F32), "rstd")
    within(n.y, y, y.abs() * (half(dtype) + 1.01 * NORM32) + last_step(dtype), "y")
    held = n.q.double() * n.scale.double()[:, None]
    within(held, y, y.abs() * (half(E4M3) + 3 * NORM32) + n.scale.double()[:, None] * 2.0 ** -10,
           "q")
    dy, dh = randn(gen(2), T, d, dtype=dtype), randn(gen(3), T, d, dtype=dtype, scale=1 / size)
    dx, dw = nm.rms_norm_backward(dy, x, n.rstd, w, dh=dh)
    clean()
    r = n.rstd.double()[:, None]
    xh, g = x.double() * r, dy.double() * w.double()
    want = r * (g - xh * (g * xh).mean(1, keepdim=True)) + dh.double()
    mag = r * (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True)) + dh.double().abs()
    within(dx, want, want.abs() * half(dtype) + mag * (85 + 8) * U + 4 * last_step(dtype), "dx")
    prod = dy.double() * xh
    within(dw, prod.sum(0), prod.abs().sum(0) * (T + 64) * U, "dweight")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,d", [(2, 64), (2, 520), (1300, 512)])
def test_norm_of_the_largest_and_the_smallest_rows(T, d, dtype):
    sign = torch.where(torch.rand(T, d, device="cuda", generator=gen(1)) < 0.5, -1.0, 1.0)
    # rstd is subnormal: half its step is 2^-150 of a value of 2^-128 or more
    x = (3e38 * sign).to(dtype)
    n = nm.rms_norm(x, eps=0.0, out="both")
    clean()
    rstd, y = norm_ref(x, None, 0.0)
    within(n.rstd, rstd, rstd * NORM32 + last_step(F32), "rstd")
    within(n.y, y, y.abs() * (half(dtype) + NORM32 + 2.0 ** -21), "y")
    # 1 / rms is beyond fp32, and rstd infinite; y is still what it is
    x = (1e-40 * sign).to(dtype)
    n = nm.rms_norm(x, eps=0.0, out="both")
    clean()
    assert bool((x != 0).all()) and bool((n.rstd == float("inf")).all())
    _, y = norm_ref(x, None, 0.0)
    within(n.y, y, y.abs() * (half(dtype) + NORM32), "y")
    # the formula's 0 / 0
    n = nm.rms_norm(torch.zeros_like(x), eps=0.0)
    clean()
    assert bool(n.y.isnan().all())


def test_norm_gradient_of_a_row_that_is_zero_in_part():
    # the mean of g xhat times rstd is beyond fp32; where h is 0 the gradient is rstd g
    d = 520
    h = torch.zeros(3, d, device="cuda")
    h[:, ::2] = 1e-37
    dy = torch.ones(3, d, device="cuda")
    dy[:, ::2] = 50.0
    rstd = nm.rms_norm(h, eps=0.0).rstd
    dx, _ = nm.rms_norm_backward(dy, h, rstd)
    clean()
    r = rstd.double()[:, None]
    xh = h.double() * r
    want = r * (dy.double() - xh * (dy.double() * xh).mean(1, keepdim=True))
    mag = r * (dy.double() + xh * (dy.double() * xh).mean(1, keepdim=True))
    within(dx, want, want.abs() * half(F32) + mag * (85 + 8) * U)


# ---- 8-bit rows ---------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,d", [(3, 8), (700, 1032), (2000, 512), (5, 16384)])
@pytest.mark.parametrize("size", [3.0, 1e-18, 1e-30, 1e-36, 1e-38, 1e30, 5e37])
def test_codes_are_those_of_the_quotient(T, d, dtype, size):
    # q = e4m3(x / scale): the code that the quotient in fp32 has, not a neighbour's
    x = randn(gen(T + d), T, d, dtype=F32, scale=size).to(dtype)
    x[0, 1], x[1, 2] = 0.0, -0.0
    q, scale = nm.quantize_rows(x)
    clean()
    assert torch.equal(q.view(torch.uint8),
                       (x.float() / scale[:, None]).to(E4M3).view(torch.uint8))
    # a norm's y in fp32 is what its q holds
    w = randn(gen(d), d, dtype=F32, scale=size)
    n = nm.rms_norm(randn(gen(T), T, d, dtype=F32), w, out="both")
    clean()
    assert torch.equal(n.q.view(torch.uint8),
                       (n.y / n.scale[:, None]).to(E4M3).view(torch.uint8))


def test_codes_of_rows_with_infinities():
    x = randn(gen(3), 4, 520)
    x[1, 5], x[2, 7], x[2, 9] = float("inf"), float("-inf"), float("nan")
    q, scale = nm.quantize_rows(x)
    clean()
    # finite / inf is 0 (of either sign), inf / inf and a row with a NaN are NaN
    got, want = q.float(), x.float() / scale[:, None]
    assert float(scale[1]) == float("inf") and bool(scale[2].isnan())
    assert torch.equal(got.isnan(), want.isnan())
    assert bool((got[1].nan_to_num(0) == 0).all()) and bool(got[3].isfinite().all())


# ---- products -------------------------------------------------------------------------------


@pytest.mark.parametrize("M,K,N", [(3, 16, 24), (60, 1008, 264), (200, 144, 136),
                                   (130, 4096, 64), (4700, 144, 2056)])
@pytest.mark.parametrize("bias", [False, True])
def test_scales_whose_product_leaves_fp32(M, K, N, bias):
    g = gen(M + N)

    def codes(rows):  # +-2^-9 .. 4 2^-9: sums of K products stay below K 2^-14
        v = torch.randint(1, 5, (rows, K), device="cuda", generator=g) * 2.0 ** -9
        sign = torch.rand(rows, K, device="cuda", generator=g) < 0.5
        return torch.where(sign, -v, v)

    a, b = codes(M), codes(N)
    a[::3] = 0                                     # sums of 0 times whatever the scales are
    sizes = torch.tensor([1e-30, 1e-10, 1.0, 1e20, 1e30, 2.0 ** -126], device="cuda")
    sx = sizes[torch.arange(M, device="cuda") % 6].contiguous()
    sw = (sizes * 0.5)[torch.arange(N, device="cuda") // 3 % 6].contiguous()
    far = (sx[:, None].double() * sw.double()) > 1e39     # only rows of 0 may meet these
    a[(far.any(1))] = 0
    bb = randn(g, N) if bias else None
    out = nm.linear_fp8(a.to(E4M3), sx, b.to(E4M3), sw, bb, out_f32=True)
    clean()
    x, w = a.double() * sx.double()[:, None], (b.double() * sw.double()[:, None]).t()
    z = x @ w
    err = product_error(x, w) + z.abs() * 3 * U
    if bias:
        z = z + bb.double()
    within(out, z, err + z.abs() * U + 2 * last_step(F32), "out")


@pytest.mark.parametrize("M,K,N", [(3, 32, 24), (200, 160, 136), (4700, 144, 2056)])
def test_small_and_large_scales_of_one_product(M, K, N):
    # both small: their product is subnormal or 0, the result is not; both large: it is beyond
    # fp32, the result is not
    g = gen(M)
    for sizes, code in (((2e-25, 3e-15), 384.0), ((2e-22, 3e-24), 448.0), ((2e21, 3e18), 2.0 ** -9),
                        ((1e-38, 2e30), 1.0), ((2.0 ** 119, 2.0 ** -126), 448.0)):
        a = (code * (1 - 2 * torch.randint(0, 2, (M, K), device="cuda", generator=g))).float()
        b = torch.full((N, K), code, device="cuda")
        b[:, 5:] = 0
        sx = torch.full((M,), sizes[0], device="cuda")
        sw = torch.full((N,), sizes[1], device="cuda")
        out = nm.linear_fp8(a.to(E4M3), sx, b.to(E4M3), sw, out_f32=True)
        clean()
        x, w = a.double() * sx.double()[:, None], (b.double() * sw.double()[:, None]).t()
        z = x @ w
        within(out, z, product_error(x, w) + z.abs() * 3 * U + last_step(F32), str(sizes))


@pytest.mark.parametrize("M,K,N", FP8_SHAPES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("f32", [False, True])
def test_linear_fp8_with_the_other_activations(M, K, N, act, f32):
    g = gen(M + K + N + 1)
    qx, sx = nm.quantize_rows(randn(g, M, K))
    qw, sw = nm.quantize_rows(randn(g, N, K, scale=K ** -0.5))
    b, r = randn(g, N), randn(g, M, N)
    out = nm.linear_fp8(qx, sx, qw, sw, b, act=act, residual=r, out_f32=f32)
    clean()
    x, w = qx.double() * sx.double()[:, None], (qw.double() * sw.double()[:, None]).t()
    z = x @ w + b.double()
    check_linear(out, z, product_error(x, w) + z.abs() * 5 * U, act, r, "out")


def activation_error(z, act):
    """The relative error of an activation in fp32. An exponential's argument is a product
    of roundings (half a step each), so its error grows with the argument as it would if z
    were moved by a few half steps; exponential and reciprocal are off by 2 ulp (2^-22) and
    one (2^-23), and the products behind them by half a step."""
    z = z.abs()
    if act == "silu":      # argument -z log2 e: the constant and the product
        return z * 2 * U + 8 * U
    if act == "gelu_tanh":  # 2 u = z (c z^2 + c'): three constants and four products, log2 e
        return 8 * U * (1.5957692 * (z + 0.044715 * z ** 3)) + 8 * U
    # x = z / sqrt 2 (two), its square (four), the sum with the fit (one), log2 e (two); the
    # fit's own 1.2e-7, its Horner steps (ten, of values below 2), the reciprocal's 2 in it
    # with a slope below 3, in the factor t, the exponential's 4, two products
    return 9 * U * (z * z / 2 + 1.3) + 1.2e-7 + (20 + 6 + 2 + 4 + 2) * U


# few rows over a cluster and in swapped tiles, whole tiles, parts over a cluster, pairs
@pytest.mark.parametrize("M,K,N", [(8, 64, 4096), (16, 2048, 512), (200, 256, 136),
                                   (100, 4096, 72), (8192, 64, 2048)])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activations_hold_their_relative_error_on_both_tails(M, K, N, act):
    g = gen(M + K)
    x = torch.zeros(M, K, dtype=BF, device="cuda")
    x[torch.arange(M), torch.arange(M) % K] = 1.0          # the product is a row of W, exactly
    w = torch.empty(K, N, device="cuda")
    w[::2] = 110 * (2 * torch.rand(w[::2].shape, device="cuda", generator=g) - 1)
    w[1::2] = 6 * torch.randn(w[1::2].shape, device="cuda", generator=g)
    w = w.to(BF)
    out = nm.linear(x, w, act=act, out_f32=True)
    clean()
    z = w.double()[torch.arange(M, device="cuda") % K]
    if act == "silu":       # (each without the cancellation of 1 + .. on the lower tail)
        want = z * torch.sigmoid(z)
    elif act == "gelu":
        want = z * torch.special.erfc(-z * 0.5 ** 0.5) / 2
    else:
        want = z * torch.sigmoid(math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3))
    # an exponential's result below 2^-126 is taken as 0
    within(out, want, want.abs() * activation_error(z, act) + z.abs() * TINY, act)
