"""The fp64 reference of the operators around a block against closed forms and
differences (CPU)."""
import math

import pytest
import torch

from oracle import block as ref


def rnd(seed):
    gen = torch.Generator().manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=gen, dtype=torch.float64)


def test_recurrence_of_constant_gates_is_a_power():
    n = rnd(1)
    C, T = 3, 9
    A, b, h0 = n(C), n(C), n(1, C)
    g, i = n(C).expand(1, T, C), torch.zeros(1, T, C, dtype=torch.float64)
    o, f = ref.scan(torch.zeros(1, T, C, dtype=torch.float64), g, i, A, b, h0)
    L = A.exp() * torch.log1p(torch.exp(g[0, 0] + b))
    for t in range(T):
        assert torch.allclose(o[0, t], h0[0] * torch.exp(-L * (t + 1)), rtol=1e-12)
    assert torch.equal(f[0], o[0, -1])


def test_recurrence_keeps_the_size_of_its_input():
    """With a gate that is open and inputs of one, h tends to sqrt(1 - a^2) / (1 - a)."""
    C = 2
    A = torch.tensor([0.0, -1.0], dtype=torch.float64)
    x = torch.ones(1, 4000, C, dtype=torch.float64)
    o, _ = ref.scan(x, torch.zeros_like(x), 60 * x, A, torch.zeros(C, dtype=torch.float64))
    a = torch.exp(-A.exp() * math.log(2.0))
    assert torch.allclose(o[0, -1], torch.sqrt(1 - a * a) / (1 - a), rtol=1e-10)


@pytest.mark.parametrize("cu", [None, [0, 3, 3, 4, 9]])
def test_recurrence_gradients_against_differences(cu):
    n = rnd(3)
    B, T, C = (2, 5, 3) if cu is None else (1, 10, 3)
    N = B if cu is None else len(cu) - 1
    args = [n(B, T, C), n(B, T, C), n(B, T, C), n(C), n(C), n(N, C)]
    for t in args:
        t.requires_grad_()
    assert torch.autograd.gradcheck(lambda *a: ref.scan(*a, cu=cu), args, atol=1e-7)
    do, df = n(B, T, C), n(N, C)
    r = ref.scan_all(*args, cu=cu, do=do, dfinal=df)
    o, f = ref.scan(*args, cu=cu)
    want = torch.autograd.grad((o * do).sum() + (f * df).sum(), args)
    for name, w in zip(("x", "g", "i", "A_log", "dt_bias", "h0"), want):
        if cu is None or name in ("A_log", "dt_bias", "h0"):
            assert torch.allclose(r[name][0], w), name
        else:
            assert torch.allclose(r[name][0][:, :cu[-1]], w[:, :cu[-1]]), name
            assert not r[name][0][:, cu[-1]:].any()
    # without an initial state its gradient is still a recurrence
    zero = torch.zeros(N, C, dtype=torch.float64)
    a = [t.detach() for t in args[:5]]
    none, some = ref.scan_all(*a, cu=cu, do=do, dfinal=df), ref.scan_all(*a, zero, cu=cu, do=do, dfinal=df)
    assert torch.allclose(none["h0"][0], some["h0"][0])


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("act", ["silu", "none"])
def test_convolution_is_a_sum_over_the_last_tokens(W, act):
    n = rnd(5)
    B, T, C = 2, 6, 3
    x, w, b, h0 = n(B, T, C), n(C, W), n(C), n(B, W - 1, C)
    y, f, _ = ref.conv(x, w, b, act, h0)
    for r in range(B):
        for t in range(T):
            for c in range(C):
                z = b[c]
                for j in range(W):
                    at = t - W + 1 + j
                    z = z + w[c, j] * (x[r, at, c] if at >= 0 else h0[r, W - 1 + at, c])
                want = z / (1 + math.exp(-z)) if act == "silu" else z
                assert abs(y[r, t, c] - want) < 1e-12
        assert torch.equal(f[r], x[r, T - W + 1:])


@pytest.mark.parametrize("cu", [None, [0, 1, 1, 3, 8]])
def test_convolution_gradients_against_differences(cu):
    n = rnd(7)
    B, T, C, W = (2, 5, 2, 4) if cu is None else (1, 9, 2, 4)
    N = B if cu is None else len(cu) - 1
    args = [n(B, T, C), n(C, W), n(C), n(N, W - 1, C)]
    for t in args:
        t.requires_grad_()
    assert torch.autograd.gradcheck(lambda x, w, b, h: ref.conv(x, w, b, "silu", h, cu)[:2], args, atol=1e-7)
    dy, df = n(B, T, C), n(N, W - 1, C)
    r = ref.conv_all(*args[:3], "silu", args[3], cu, dy, df)
    y, f, _ = ref.conv(*args[:3], "silu", args[3], cu)
    want = torch.autograd.grad((y * dy).sum() + (f * df).sum(), args)
    for name, v in zip(("dweight", "dbias", "dh0"), want[1:]):
        assert torch.allclose(r[name][0], v), name


def test_layer_norm_against_differences_and_its_moments():
    n = rnd(9)
    u, w, b = 3 * n(4, 8) + 2, n(8), n(8)
    y = ref.layer_norm(u, torch.ones(8, dtype=torch.float64), None, 0.0)
    assert torch.allclose(y.mean(-1), torch.zeros(4, dtype=torch.float64), atol=1e-12)
    assert torch.allclose((y * y).mean(-1), torch.ones(4, dtype=torch.float64))
    args = [u.requires_grad_(), w.requires_grad_(), b.requires_grad_()]
    assert torch.autograd.gradcheck(lambda *a: ref.layer_norm(*a), args, atol=1e-7)
    assert torch.allclose(ref.layer_norm(u, w, b), torch.nn.functional.layer_norm(u, (8,), w, b, 1e-5))
