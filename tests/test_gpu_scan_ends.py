"""The gated linear recurrence where a gate, a state or a gradient leaves the usual range:
gradients of fixed lengths that fill no tile."""
import pytest
import torch

from block_util import near
from oracle import block as ref
from test_gpu_scan import args, make, run

pytestmark = pytest.mark.gpu
GRADS = (("dx", "x"), ("dg", "g"), ("dinput_gate", "i"), ("dh0", "h0"), ("dA_log", "A_log"), ("ddt_bias", "dt_bias"))
INF = float("inf")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 9, 63, 64, 70, 300])
def test_a_channel_that_forgets_everything_at_any_length(T, dtype):
    """dt_bias = +inf: the decay is zero, and so is every gradient through it.  In 64 bits
    it is zero from a dt_bias of 1e6 on, with which the reference has no infinity."""
    w = make(2, T, 24, seed=101, dtype=dtype)
    w["A_log"][5] = 0.0
    w["dt_bias"][5] = INF
    o, f, r = run(w)
    w["dt_bias"][5] = 1e6
    want = ref.scan_all(*args(w), w["h0"], None, w["do"], w["dfinal"])
    near("o", o, want["o"])
    near("final", f, want["final"])
    for got, name in GRADS[:4]:
        near(got, r[got], want[name])
    near("ddt_bias", r["ddt_bias"], want["dt_bias"])
    assert not r["dg"][..., 5].any() and not r["dh0"][:, 5].any()


@pytest.mark.parametrize("T", [3, 70])
def test_a_large_gradient_of_the_last_state_meets_a_large_state(T):
    """Their product is beyond fp32, but nothing of it belongs to a token: the last decay
    brings it back, and the rows behind the last token have none."""
    w = make(2, T, 24, seed=103, dtype="fp32")
    w["x"] *= 2.0 ** 40
    w["h0"] *= 2.0 ** 40
    w["dfinal"] *= 2.0 ** 100
    w["gate"][:] = 30.0  # (its own gradient stays in fp32's range)
    w["A_log"][:] = 0.0
    w["dt_bias"][:] = 30.0
    w["g"][:] = torch.linspace(-1.0, 1.0, 24)
    _, _, r = run(w)
    want = ref.scan_all(*args(w), w["h0"], None, w["do"], w["dfinal"])
    for got, name in GRADS:
        near(got, r[got], want[name])
