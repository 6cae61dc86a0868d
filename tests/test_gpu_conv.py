"""GPU parity of the short causal convolution (short_conv_fwd, short_conv_bwd,
short_conv_decode, short_conv) against the fp64 sums.

Tolerances: one rounding to the tokens' type, and the reference's bound: 8 * 2^-24
of the absolute terms of a sum over taps, 2^-20 for the activation, 2^-18 of the
absolute sum for sums over tokens."""
import pytest
import torch

import chunked_gated_delta_kda_amd as kda
from block_util import DEV, TYPES, near, offsets, to_gpu
from oracle import block as ref
from parity_util import say
from test_gpu_graph import REPLAYS, capture

pytestmark = pytest.mark.gpu


def make(B, T, C, W=4, seed=1, dtype="bf16", bias=True, init=True, cu=None, act="silu"):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    N = B if cu is None else len(cu) - 1
    tt = TYPES[dtype]
    return dict(x=n(B, T, C).to(tt), weight=n(C, W), bias=n(C) if bias else None, act=act,
                h0=n(N, W - 1, C).to(tt) if init else None, cu=cu, dy=n(B, T, C).to(tt),
                dfinal=n(N, W - 1, C).to(tt))


def run(w):
    d = to_gpu(w)
    y, f = kda.short_conv_fwd(d["x"], d["weight"], d["bias"], d["act"], d["h0"], cu_seqlens=d["cu"])
    r = kda.short_conv_bwd(d["x"], d["weight"], d["dy"], d["bias"], d["act"], d["h0"], d["dfinal"], d["cu"])
    return y, f, r


def check(w):
    y, f, r = run(w)
    torch.cuda.synchronize()
    say(f"[conv] {tuple(w['x'].shape)} {w['x'].dtype} W {w['weight'].shape[1]} {w['act']} packed {w['cu'] is not None}")
    h0 = w["h0"]
    zero = torch.zeros_like(w["dfinal"])
    want = ref.conv_all(w["x"], w["weight"], w["bias"], w["act"], zero if h0 is None else h0, w["cu"], w["dy"],
                        w["dfinal"])
    near("y", y, want["y"])
    assert torch.equal(f.double().cpu(), want["final"][0])
    for n in ("dx", "dweight", "dh0") + (("dbias",) if w["bias"] is not None else ()):
        near(n, r[n], want[n])
    assert (r["dbias"] is None) == (w["bias"] is None)
    return y, f, r


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 31, 32, 33, 35, 129])
def test_lengths(T, W, dtype):
    check(make(2, T, 24, W, seed=T, dtype=dtype))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("C", [8, 248, 256, 264, 512, 520, 1032])
def test_channels(C, dtype):
    check(make(1, 40, C, seed=C, dtype=dtype))


@pytest.mark.parametrize("bias,init,act", [(True, False, "silu"), (False, True, "none"), (False, False, "none"),
                                           (False, False, "silu")])
def test_parts(bias, init, act):
    check(make(3, 70, 40, seed=5, bias=bias, init=init, act=act))


LENS = [[5], [0, 5, 0], [1, 1, 1, 2, 3, 130], [32, 31, 1, 128, 1, 0, 0, 3], [300, 0, 17], [0, 0], [1] * 70, [2] * 40]


@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("tail", [0, 21, 150])
@pytest.mark.parametrize("lens", LENS)
def test_packed(lens, tail, dtype, W):
    cu = offsets(lens)
    T = int(cu[-1]) + tail
    if T == 0:
        pytest.skip("no rows: test_no_tokens")
    w = make(1, T, 40, W, seed=len(lens), dtype=dtype, cu=cu)
    for n in ("x", "dy"):
        w[n][:, int(cu[-1]):] = float("nan")
    y, _, r = check(w)
    assert not y[:, int(cu[-1]):].any() and not r["dx"][:, int(cu[-1]):].any()


def test_packed_that_begins_late():
    cu = torch.tensor([20, 150, 150, 290], dtype=torch.int32)
    y, _, r = check(make(1, 300, 64, seed=11, cu=cu))
    assert not y[:, :20].any() and not r["dx"][:, :20].any() and not y[:, 290:].any()


def test_packed_is_each_sequence_by_itself():
    lens = [200, 1, 77, 2, 256, 5]
    cu = offsets(lens)
    w = make(1, int(cu[-1]), 128, seed=13, cu=cu)
    d = to_gpu(w)
    y, f = kda.short_conv_fwd(d["x"], d["weight"], d["bias"], "silu", d["h0"], cu_seqlens=d["cu"])
    for n, (a, e) in enumerate(zip(cu[:-1].tolist(), cu[1:].tolist())):
        y1, f1 = kda.short_conv_fwd(d["x"][:, a:e].contiguous(), d["weight"], d["bias"], "silu",
                                    d["h0"][n:n + 1].contiguous())
        assert torch.equal(y[:, a:e], y1) and torch.equal(f[n:n + 1], f1)


def test_nan_stays_in_the_tokens_that_see_it():
    cu = offsets([50, 40, 60])
    w = make(1, 150, 72, seed=19, cu=cu)
    y, f, r = run(w)
    w["x"][0, 48, 5] = float("nan")
    w["dy"][0, 70, 9] = float("nan")
    y2, f2, r2 = run(w)
    clean = torch.ones(150, 72, dtype=torch.bool, device=DEV)
    clean[48:50, 5] = False
    assert torch.equal(y[0][clean], y2[0][clean]) and y2[0, 48:50, 5].isnan().all()
    assert torch.equal(f[1:], f2[1:])
    clean[45:50, 5] = False
    clean[67:71, 9] = False
    assert torch.equal(r["dx"][0][clean], r2["dx"][0][clean])
    ok = torch.ones(72, dtype=torch.bool, device=DEV)
    ok[[5, 9]] = False
    assert torch.equal(r["dweight"][ok], r2["dweight"][ok]) and torch.equal(r["dbias"][ok], r2["dbias"][ok])


def test_activations_at_the_ends():
    """silu(-90) is -7.4e-38, and its slope is of the same kind."""
    w = make(1, 20, 16, seed=21, dtype="fp32", init=False, bias=False)
    w["weight"][:] = 0.0
    w["weight"][:, -1] = 1.0
    w["x"][:] = torch.linspace(-87.0, 87.0, 20 * 16).view(1, 20, 16)
    y, _, r = run(w)
    z = w["x"].double()
    want = z / (1 + torch.exp(-z))
    assert ((y.double().cpu() - want).abs() <= 2.0 ** -18 * want.abs() + 2.0 ** -126).all()


@pytest.mark.parametrize("packed", [False, True])
def test_no_tokens(packed):
    cu = torch.zeros(4, dtype=torch.int32) if packed else None
    w = make(1 if packed else 3, 0, 16, seed=23, cu=cu)
    y, f, r = run(w)
    assert y.numel() == 0 and torch.equal(f.cpu(), w["h0"]) and torch.equal(r["dh0"].cpu(), w["dfinal"])
    assert not r["dweight"].any() and not r["dbias"].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("N,C", [(1, 8), (5, 360), (64, 4096)])
def test_decode_continues_the_forward_pass(N, C, W, dtype):
    w = make(N, 9, C, W, seed=C, dtype=dtype)
    d = to_gpu(w)
    y, f = kda.short_conv_fwd(d["x"], d["weight"], d["bias"], "silu", d["h0"])
    _, state = kda.short_conv_fwd(d["x"][:, :8].contiguous(), d["weight"], d["bias"], "silu", d["h0"])
    tok = d["x"][:, 8].contiguous()
    before = state.clone()
    y1, new = kda.short_conv_decode(tok, d["weight"], state, d["bias"])
    assert torch.equal(y1, y[:, 8]) and torch.equal(new, f) and torch.equal(state, before)
    y2, new2 = kda.short_conv_decode(tok, d["weight"], state, d["bias"], state_out=state)
    assert new2 is state and torch.equal(y2, y1) and torch.equal(state, new)


def test_equal_calls_give_equal_bits():
    w = make(2, 1000, 264, seed=29)
    a, b = run(w), run(w)
    assert torch.equal(a[0], b[0]) and all(torch.equal(a[2][n], b[2][n]) for n in a[2])


def test_autograd_is_short_conv_bwd():
    cu = offsets([70, 0, 30])
    w = make(1, 100, 64, seed=31, cu=cu)
    d = to_gpu(w)
    lv = {n: d[n].clone().requires_grad_() for n in ("x", "weight", "bias", "h0")}
    y, f = kda.short_conv(lv["x"], lv["weight"], lv["bias"], "silu", lv["h0"], True, d["cu"])
    got = torch.autograd.grad([y, f], list(lv.values()), [d["dy"], d["dfinal"]])
    _, _, r = run(w)
    for a, n in zip(got, ("dx", "dweight", "dbias", "dh0")):
        assert torch.equal(a, r[n]), n
    (gx,) = torch.autograd.grad(kda.short_conv(lv["x"], lv["weight"], lv["bias"], "silu", lv["h0"], True,
                                               d["cu"])[1], [lv["x"]], d["dfinal"])
    assert torch.equal(gx, run({**w, "dy": torch.zeros_like(w["dy"])})[2]["dx"])


def test_graph_replays_equal_eager():
    w = make(1, 300, 128, seed=37)
    y0, f0, r0 = run(w)
    d = to_gpu(w)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    res = {}

    def call():
        res["y"], res["f"] = kda.short_conv_fwd(d["x"], d["weight"], d["bias"], "silu", d["h0"])
        res.update(kda.short_conv_bwd(d["x"], d["weight"], d["dy"], d["bias"], "silu", d["h0"], d["dfinal"],
                                      workspace=ws))

    g = capture(call)
    for _ in range(REPLAYS):
        for t in res.values():
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for n, t in dict(r0, y=y0, f=f0).items():
            assert torch.equal(res[n], t), n
