"""GPU parity of the layer norm (layer_norm_fwd, layer_norm_bwd, layer_norm)
against the fp64 formulas.

Tolerances: one rounding to the rows' type, 2^-17 of the absolute terms (fp32 sums
of up to 16384 terms over lanes), and 2^-21 of the values for the differences from
the mean."""
import pytest
import torch

import chunked_gated_delta_kda_amd as kda
from block_util import DEV, TYPES, near, to_gpu
from oracle import block as ref
from parity_util import say
from test_gpu_graph import REPLAYS, capture

pytestmark = pytest.mark.gpu


def make(shape, seed, dtype="bf16", bias=True, res=True, dsum=None, spread=1.0, mean=0.0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    D, tt = shape[-1], TYPES[dtype]
    return dict(x=(n(*shape).double() * spread + mean).to(tt), weight=n(D), bias=n(D) if bias else None,
                residual=(n(*shape).double() * spread).to(tt) if res else None, dy=n(*shape).to(tt),
                dsum=n(*shape).to(tt) if (res if dsum is None else dsum) else None)


def run(w, eps=1e-5):
    d = to_gpu(w)
    y, u = kda.layer_norm_fwd(d["x"], d["weight"], d["bias"], eps, d["residual"])
    r = kda.layer_norm_bwd(u, d["weight"], d["dy"], eps, d["dsum"], need_dbias=d["bias"] is not None)
    return y, u, r


def check(w, eps=1e-5):
    y, u, r = run(w, eps)
    torch.cuda.synchronize()
    say(f"[layer norm] {tuple(w['x'].shape)} {w['x'].dtype} residual {w['residual'] is not None}")
    if w["residual"] is None:
        assert torch.equal(u.cpu(), w["x"])
    else:
        assert torch.equal(u.cpu(), (w["x"].double() + w["residual"].double()).float().to(w["x"].dtype))
    want = ref.layer_norm_all(u, w["weight"], w["bias"], eps, w["dy"], w["dsum"])
    near("y", y, want["y"])
    for n in ("dx", "dweight") + (("dbias",) if w["bias"] is not None else ()):
        near(n, r[n], want[n])
    assert (r["dbias"] is None) == (w["bias"] is None)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [8, 16, 24, 40, 64, 72, 128, 136, 256, 264, 512, 520, 1000, 1024, 1032, 2048, 2056, 4096,
                               4104, 8192, 8200, 16384])
def test_channels(D, dtype):
    check(make((7, D), seed=D, dtype=dtype))


@pytest.mark.parametrize("bias,res,dsum", [(True, False, False), (False, True, True), (False, False, True),
                                           (False, True, False)])
def test_parts(bias, res, dsum):
    check(make((2, 33, 136), seed=7, bias=bias, res=res, dsum=dsum))


@pytest.mark.parametrize("shape", [(1, 64), (64,), (5000, 64), (3, 1, 5, 128), (1, 4096), (2500, 1032)])
def test_shapes(shape):
    check(make(shape, seed=11))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("mean", [3.0, -100.0])
def test_rows_far_from_zero(mean, dtype):
    check(make((20, 1000), seed=13, dtype=dtype, mean=mean, res=False))


@pytest.mark.parametrize("D", [72, 4096])
@pytest.mark.parametrize("spread,eps", [(1e-4, 1e-5), (0.0, 1e-5), (1e8, 0.0), (1e25, 1e-5), (1e37, 0.0),
                                        (1e-25, 0.0), (1e-18, 1e-36), (1e-30, 1e-36)])
def test_scales_of_the_rows(spread, eps, D):
    """The norm is of the size of one whatever the row's."""
    w = make((20, D), seed=17, spread=spread, res=False)
    w["dy"] = (w["dy"].double() * min(1.0, max(spread, 1e-20))).to(torch.bfloat16)  # dx in bf16's range
    check(w, eps)


def test_nan_stays_in_its_row():
    for D in (72, 4096):
        w = make((50, D), seed=19)
        y, u, r = run(w)
        w["x"][20, 5] = float("nan")
        w["residual"][30, 71] = float("inf")
        y2, u2, r2 = run(w)
        clean = torch.ones(50, dtype=torch.bool, device=DEV)
        clean[[20, 30]] = False
        assert torch.equal(y[clean], y2[clean]) and torch.equal(r["dx"][clean], r2["dx"][clean])
        assert y2[20].isnan().all() and y2[30].isnan().all()
        assert torch.equal(r["dbias"], r2["dbias"])


def test_no_rows():
    for res in (False, True):
        y, u, r = run(make((0, 64), seed=23, res=res))
        assert y.shape == (0, 64) and u.shape == (0, 64)
        assert not r["dweight"].any() and not r["dbias"].any()


def test_in_place():
    for D in (72, 1024, 4096):
        w = make((30, D), seed=29)
        y, u, _ = run(w)
        for a, b in (("x", "residual"), ("residual", "x")):
            d = to_gpu(w)
            y2, u2 = kda.layer_norm_fwd(d["x"], d["weight"], d["bias"], 1e-5, d["residual"], out=d[a], sum_out=d[b])
            assert y2 is d[a] and u2 is d[b] and torch.equal(y, y2) and torch.equal(u, u2)


def test_equal_calls_give_equal_bits():
    w = make((3000, 520), seed=31)
    a, b = run(w), run(w)
    assert torch.equal(a[0], b[0]) and all(torch.equal(a[2][n], b[2][n]) for n in a[2])


def test_autograd_is_layer_norm_bwd():
    w = make((3, 17, 136), seed=37)
    d = to_gpu(w)
    names = ("x", "weight", "bias", "residual")
    lv = {n: d[n].clone().requires_grad_() for n in names}
    y, u = kda.layer_norm(lv["x"], lv["weight"], lv["bias"], 1e-5, lv["residual"])
    got = torch.autograd.grad([y, u], [lv[n] for n in names], [d["dy"], d["dsum"]])
    _, _, r = run(w)
    for a, n in zip(got, ("dx", "dweight", "dbias", "dx")):
        assert torch.equal(a, r[n]), n
    # either output alone
    y, u = kda.layer_norm(lv["x"], lv["weight"], lv["bias"], 1e-5, lv["residual"])
    (gx,) = torch.autograd.grad(y, [lv["x"]], d["dy"], retain_graph=True)
    assert torch.equal(gx, run({**w, "dsum": None})[2]["dx"])
    (gx,) = torch.autograd.grad(u, [lv["residual"]], d["dsum"])
    assert torch.equal(gx, d["dsum"])
    # without a residual
    y, same = kda.layer_norm(lv["x"], lv["weight"])
    assert same is lv["x"]
    (gx,) = torch.autograd.grad(y, [lv["x"]], d["dy"])
    assert torch.equal(gx, run({**w, "dsum": None, "residual": None, "bias": None})[2]["dx"])


def test_graph_replays_equal_eager():
    w = make((300, 1032), seed=41)
    y0, u0, r0 = run(w)
    d = to_gpu(w)
    res = {}

    def call():
        res["y"], res["u"] = kda.layer_norm_fwd(d["x"], d["weight"], d["bias"], 1e-5, d["residual"])
        res.update(kda.layer_norm_bwd(res["u"], d["weight"], d["dy"], 1e-5, d["dsum"]))

    g = capture(call)
    for _ in range(REPLAYS):
        for t in res.values():
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for n, t in dict(r0, y=y0, u=u0).items():
            assert torch.equal(res[n], t), n
