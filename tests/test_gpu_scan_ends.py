"""The gated linear recurrence where a gate, a state or a gradient leaves the usual range:
gradients of fixed lengths that fill no tile."""
import pytest
import torch

import chunked_gated_delta_kda_amd as kda
from block_util import near, to_gpu
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


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("C", [24, 712])  # (few chains and many)
def test_tokens_that_reset_the_state(C, dtype, packed):
    """A gate of the type's largest value or of +inf, or the product of a large one and a
    large exp(A_log): L is infinite in fp32, the decay zero, and the token adds nothing to
    any gradient through its gate.  In 64 bits that is so from L = 1e6 on."""
    cu = torch.tensor([0, 40, 40, 131], dtype=torch.int32) if packed else None
    w = make(1, 139, C, seed=107, dtype=dtype, cu=cu)
    big = torch.finfo(w["g"].dtype).max
    w["A_log"][2], w["dt_bias"][2] = 3.0, -6.0
    resets = ((5, 1, big), (63, 1, INF), (64, 3, INF), (39, 4, big), (40, 4, INF), (130, 5, big), (20, 2, big / 4))
    for t, c, v in resets:
        w["g"][0, t, c] = v
    o, f, r = run(w)
    for t, c, _ in resets:
        w["g"][0, t, c] = 1e6
    want = ref.scan_all(*args(w), w["h0"], w["cu"], w["do"], w["dfinal"])
    near("o", o, want["o"])
    near("final", f, want["final"])
    for got, name in GRADS:
        near(got, r[got], want[name])
    for t, c, _ in resets:
        assert r["dg"][0, t, c] == 0


@pytest.mark.parametrize("T", [64, 70])
def test_a_channel_that_forgets_everything_has_no_gradient_of_its_decay(T):
    w = make(2, T, 24, seed=109)
    w["A_log"][5] = 0.0
    w["dt_bias"][5] = INF
    _, _, r = run(w)
    assert r["dA_log"][5] == 0 and r["ddt_bias"][5] == 0 and torch.isfinite(r["dA_log"]).all()


def test_a_nan_in_a_gate_still_reaches_its_channels_gradients():
    w = make(1, 70, 24, seed=113)
    w["g"][0, 30, 3] = float("nan")
    _, _, r = run(w)
    for n in ("dA_log", "ddt_bias"):
        assert r[n][3].isnan() and torch.isfinite(r[n][:3]).all() and torch.isfinite(r[n][4:]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 70, 300])
def test_a_channel_that_keeps_everything(T, dtype):
    """dt_bias = -inf: nothing enters and nothing is forgotten, and no gradient passes the
    gate; the initial state has the sum of the outputs' gradients."""
    w = make(2, T, 24, seed=127, dtype=dtype)
    w["dt_bias"][7] = -INF
    o, f, r = run(w)
    assert torch.equal(f[:, 7].cpu(), w["h0"][:, 7])
    assert torch.equal(o[..., 7].cpu(), w["h0"][:, None, 7].expand(2, T).to(w["x"].dtype))
    for n in ("dx", "dg", "dinput_gate"):
        assert not r[n][..., 7].any() and torch.isfinite(r[n]).all()
    assert r["dA_log"][7] == 0 and r["ddt_bias"][7] == 0
    do = w["do"][..., 7].double()
    want = do.sum(1) + w["dfinal"][:, 7]
    # a sum of T + 1 terms in fp32, 2^-24 of each partial sum
    assert ((r["dh0"][:, 7].double().cpu() - want).abs()
            <= (T + 1) * 2.0 ** -24 * (do.abs().sum(1) + w["dfinal"][:, 7].abs())).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_single_tokens_with_infinite_gates(dtype):
    w = to_gpu(make(3, 1, 16, seed=131, dtype=dtype))
    tok = [w[k][:, 0].contiguous() for k in ("x", "g", "gate")]
    w["dt_bias"][0], w["dt_bias"][1] = INF, -INF
    tok[1][:, 2], tok[1][:, 3], tok[1][:, 4] = INF, -INF, torch.finfo(tok[1].dtype).max
    o, s = kda.gated_scan_decode(*tok, w["A_log"], w["dt_bias"], w["h0"])
    assert torch.isfinite(s).all()
    assert torch.equal(s[:, [1, 3]], w["h0"][:, [1, 3]])
    forgets = [0, 2, 4]
    want = (torch.sigmoid(tok[2].double()) * tok[0].double())[:, forgets]
    assert ((s[:, forgets].double() - want).abs() <= 2.0 ** -20 * want.abs()).all()
    assert torch.equal(o, s.to(o.dtype))
