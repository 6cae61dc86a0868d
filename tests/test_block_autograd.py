"""What the differentiable wrappers around a block do with derivatives they have no rule
for (CPU: the calls of the binding are replaced)."""
import pytest
import torch
from torch.autograd import forward_ad

import chunked_gated_delta_kda_amd as kda
from chunked_gated_delta_kda_amd import autograd

B, T, C = 2, 5, 8


@pytest.fixture
def calls(monkeypatch):
    """Stand-ins for the kernels' calls; which ran, in order."""
    ran = []

    def scan(save):
        def call(x, g, gate, A, b, h0=None, final=True, cu=None):
            ran.append("save" if save else "plain")
            f = torch.zeros(B, C) if final else None
            return (x.clone(), f, torch.zeros(8)) if save else (x.clone(), f)
        return call

    def conv(x, weight, bias, act, h0, final, cu):
        return x.clone(), torch.zeros(B, 3, C) if final else None

    def norm(x, weight, bias, eps, residual):
        return x.clone(), x if residual is None else x + residual

    monkeypatch.setattr(autograd._b, "gated_scan_fwd_save", scan(True))
    monkeypatch.setattr(autograd._b, "gated_scan_fwd", scan(False))
    monkeypatch.setattr(autograd._b, "short_conv_fwd", conv)
    monkeypatch.setattr(autograd._b, "layer_norm_fwd", norm)
    return ran


def wrappers(x):
    p, taps = torch.zeros(C), torch.zeros(C, 4)
    return {"scan": lambda: kda.gated_scan(x, x, x, p, p)[0],
            "scan with its state": lambda: kda.gated_scan(x, x, x, p, p, output_final_state=True)[0],
            "conv": lambda: kda.short_conv(x, taps)[0],
            "norm": lambda: kda.layer_norm(x, p)[0],
            "norm with a skip": lambda: kda.layer_norm(x, p, residual=x)[0]}


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("name", list(wrappers(None)))
def test_a_tangent_is_refused_not_dropped(calls, name, grad):
    x, t = torch.randn(B, T, C), torch.randn(B, T, C)
    with torch.set_grad_enabled(grad), forward_ad.dual_level():
        with pytest.raises(NotImplementedError):
            wrappers(forward_ad.make_dual(x, t))[name]()


@pytest.mark.parametrize("name", list(wrappers(None)))
def test_a_batched_tensor_is_refused(calls, name):
    with pytest.raises(RuntimeError):
        torch.func.vmap(lambda x: wrappers(x)[name]())(torch.randn(3, B, T, C))


@pytest.mark.parametrize("final", [True, False])
def test_states_are_kept_only_where_a_gradient_is_recorded(calls, final):
    p, x = torch.zeros(C), torch.randn(B, T, C)
    leaf = x.clone().requires_grad_()
    o, f = kda.gated_scan(x, x, x, p, p, output_final_state=final)
    assert not o.requires_grad and (f is None) != final
    with torch.no_grad():
        o, f = kda.gated_scan(leaf, x, x, p, p, output_final_state=final)
    assert not o.requires_grad and (f is None) != final
    assert calls == ["plain", "plain"]
    for leaves in ((leaf, x, p), (x, leaf, p), (x, x, p.clone().requires_grad_())):
        o, f = kda.gated_scan(leaves[0], x, leaves[1], leaves[2], p, output_final_state=final)
        assert o.requires_grad and (f is None) != final
    assert calls[2:] == ["save"] * 3


def test_a_sum_that_would_not_be_written_is_refused():
    x, p = torch.zeros(4, C), torch.zeros(C)
    with pytest.raises(ValueError, match="residual"):
        kda.layer_norm_fwd(x, p, sum_out=torch.zeros(4, C))
