"""The convolution's silu and its slope where the sigmoid leaves fp32's normal numbers.

With one tap of weight one z is x itself.  The kernel's sigmoid of a negative z is e^-|z| =
h h with h = 2^(-|z| / (2 ln 2)): the exponent, at most 75, is off by its own rounding and
that of the product it comes from, 2^-23 of it together, and so is h, twice that with the
logarithm of two the square (|z| 2^-23), and a few ulps more (2^-20).  What is left below the
normal numbers is rounded to steps of 2^-149, in e, in what it is multiplied to and in the
output: |z| + 2 half steps."""
import math

import pytest
import torch

import chunked_gated_delta_kda_amd as kda
from block_util import DEV, TYPES

pytestmark = pytest.mark.gpu
T, C = 105, 64


def z64():
    return torch.linspace(-104.0, 104.0, T * C, dtype=torch.float64).view(1, T, C)


def inputs(dtype):
    x = z64().to(TYPES[dtype])
    w = torch.zeros(C, 4)
    w[:, -1] = 1.0
    return x, w, x.double()


def last(dtype):
    """The type's smallest number: 2^-149, bf16 2^-133 (half of it and less is zero: silu(-98)
    in bf16)."""
    return torch.finfo(TYPES[dtype]).smallest_normal * torch.finfo(TYPES[dtype]).eps


def there(z, want, dtype):
    """Where neither the output nor e^-|z| (fp32, zero below 2^-150) may round to zero."""
    return (z < 0) & (want.abs() > 2 * last(dtype)) & (z.abs() < 150 * math.log(2.0) - 1)


def tolerance(z, terms, dtype):
    """terms: the absolute values that are added up."""
    half = torch.finfo(TYPES[dtype]).eps / 2
    return terms * (z.abs() * 2.0 ** -23 + 2.0 ** -20 + half * 1.01) + (z.abs() + 2) * 2.0 ** -150 + last(dtype) / 2


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_silu_down_to_its_last_number(dtype):
    x, w, z = inputs(dtype)
    want = z / (1 + torch.exp(-z))
    y, _ = kda.short_conv_fwd(x.to(DEV), w.to(DEV))
    one, _ = kda.short_conv_decode(x[0].to(DEV), w.to(DEV), torch.zeros(T, 3, C, dtype=x.dtype, device=DEV))
    for got in (y.double().cpu(), one.double().cpu()[None]):
        assert ((got - want).abs() <= tolerance(z, want.abs(), dtype)).all()
    # numbers below the normal ones are there: silu(-92) is -1.0e-38
    below = (want.abs() < 2.0 ** -126) & there(z, want, dtype)
    assert below.any() and (y.cpu()[below] < 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_its_slope_down_to_its_last_number(dtype):
    x, w, z = inputs(dtype)
    s = 1 / (1 + torch.exp(-z))
    rest = 1 / (1 + torch.exp(z))  # 1 - s
    want = s + z * s * rest
    terms = s + (z * s * rest).abs()
    r = kda.short_conv_bwd(x.to(DEV), w.to(DEV), torch.ones_like(x).to(DEV))
    got = r["dx"].double().cpu()
    assert ((got - want).abs() <= tolerance(z, terms, dtype)).all()
    below = (want.abs() < 2.0 ** -126) & there(z, want, dtype)
    assert below.any() and (r["dx"].cpu()[below] < 0).all()
    # the tap's own gradient: the sum over tokens of x times the slope
    assert ((r["dweight"][:, -1].double().cpu() - (z * want).sum((0, 1))).abs()
            <= (z.abs() * (tolerance(z, terms, "fp32"))).sum((0, 1)) + 2.0 ** -18 * (z * want).abs().sum((0, 1))).all()


def test_a_nan_is_one():
    x, w, _ = inputs("fp32")
    x[0, 50] = float("nan")
    y, _ = kda.short_conv_fwd(x.to(DEV), w.to(DEV))
    r = kda.short_conv_bwd(x.to(DEV), w.to(DEV), torch.ones_like(x).to(DEV))
    assert y[0, 50].isnan().all() and r["dx"][0, 50].isnan().all() and r["dweight"].isnan().all()
