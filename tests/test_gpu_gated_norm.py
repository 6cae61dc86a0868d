"""GPU parity of the gated norm (gated_norm_fwd, gated_norm_bwd, gated_norm) and
of the layer it ends, against the fp64 formulas.

Tolerances: everything is fp32 up to one rounding to bf16 (2^-8 of the value);
fp32 sums of up to 512 terms, products of up to eight factors and the
exponential are off by less than 2^-17 of the terms' absolute sum.  Sums over
rows (dweight, dresidual_scale) are fp32 terms added up in fp32 within a
workgroup and in 64 bits over them: 2^-16 of the absolute sum."""
import numpy as np
import pytest
import torch

import chunked_gated_delta_kda_amd as kda
from oracle import linear as ref
from parity_util import say
from test_gpu_graph import REPLAYS, capture

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FINE = 2.0 ** -17


def make(shape, seed, gated=True, res=True, spread=1.0):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    H, D = shape[-2:]
    bf = torch.bfloat16
    return dict(x=(n(*shape) * spread).to(bf), gate=(2 * n(*shape)).to(bf) if gated else None, weight=n(D),
                residual=n(*shape).to(bf) if res else None, residual_scale=n(H) if res else None,
                dy=n(*shape).to(bf))


def run(w, act, eps=1e-6, **kw):
    d = {k: None if t is None else t.to(DEV) for k, t in w.items()}
    a = (d["x"], d["gate"], d["weight"])
    k = dict(activation=act, eps=eps, residual=d["residual"], residual_scale=d["residual_scale"])
    y = kda.gated_norm_fwd(*a, **k)
    return y, kda.gated_norm_bwd(*a, d["dy"], **k)


def check(w, act, eps=1e-6):
    say(f"[norm] {tuple(w['x'].shape)} {act} gate {w['gate'] is not None} residual {w['residual'] is not None}")
    y, r = run(w, act, eps)
    torch.cuda.synchronize()
    c = {k: None if t is None else t.double() for k, t in w.items()}
    want = ref.gated_norm(c["x"], c["gate"], c["weight"], act, eps, c["residual"], c["residual_scale"], c["dy"])
    c = {k: None if t is None else t.numpy() for k, t in c.items()}
    u = c["x"] if c["residual"] is None else c["x"] + c["residual_scale"][:, None] * c["residual"]
    ua = np.abs(c["x"]) + (0 if c["residual"] is None else np.abs(c["residual_scale"][:, None] * c["residual"]))
    root = np.sqrt((u * u).mean(-1, keepdims=True) + eps)
    z = c["gate"]
    s = 1 if z is None else 1 / (1 + np.exp(-z))
    act_a = s if act == "sigmoid" or z is None else np.abs(z) * s
    slope_a = 0 if z is None else s * (1 + np.abs(z)) if act == "silu" else s
    n_a, t_a = ua / root, np.abs(c["dy"] * c["weight"]) * act_a
    dx_a = (t_a + n_a * (t_a * n_a).mean(-1, keepdims=True)) / root
    mags = dict(y=n_a * np.abs(c["weight"]) * act_a, dx=dx_a, dgate=np.abs(c["dy"] * c["weight"]) * n_a * slope_a)
    got = dict(r, y=y)
    if c["residual"] is not None:
        mags["dresidual"] = dx_a * np.abs(c["residual_scale"][:, None])
    for n, mag in mags.items():
        if got[n] is None:
            assert z is None and n == "dgate"
            continue
        g = got[n].double().cpu().numpy()
        assert np.all(np.isfinite(g)), n
        bad = np.abs(g - want[n]) - 2.0 ** -8 * np.abs(want[n]) - FINE * mag - 1e-37
        assert bad.max() <= 0, (n, bad.max())
    rows = tuple(range(u.ndim - 1))
    sums = dict(dweight=(np.abs(c["dy"]) * n_a * act_a).sum(rows))
    if c["residual"] is not None:
        sums["dresidual_scale"] = (dx_a * np.abs(c["residual"])).sum(rows[:-1] + (u.ndim - 1,))
    for n, mag in sums.items():
        g = got[n].double().cpu().numpy()
        assert np.all(np.abs(g - want[n]) <= 2 * FINE * mag), (n, np.abs(g - want[n]).max())


@pytest.mark.parametrize("D", [8, 16, 24, 40, 64, 72, 128, 136, 256, 264, 512])
def test_channels(D):
    check(make((7, 3, D), seed=D), "silu")


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("gated,res", [(True, True), (True, False), (False, True), (False, False)])
def test_parts(act, gated, res):
    check(make((2, 33, 5, 128), seed=7, gated=gated, res=res), act)


@pytest.mark.parametrize("shape", [(1, 1, 64), (1, 64), (5000, 7, 64), (3, 1, 4, 128)])
def test_shapes(shape):
    check(make(shape, seed=11), "sigmoid")


@pytest.mark.parametrize("spread,eps", [(1e-4, 1e-6), (1e-18, 1e-6), (0.0, 1e-6), (1e8, 0.0)])
def test_scales_of_the_rows(spread, eps):
    check(make((40, 2, 128), seed=13, spread=spread, res=False), "silu", eps)


def test_gates_at_the_ends():
    w = make((16, 2, 64), seed=17, res=False)
    w["gate"][:, 0] = 120.0
    w["gate"][:, 1] = -120.0
    for act in ("sigmoid", "silu"):
        check(w, act)


def test_nan_stays_in_its_row():
    w = make((50, 3, 72), seed=19)
    y, r = run(w, "silu")
    w["x"][20, 1, 5] = float("nan")
    w["gate"][30, 2, 71] = float("inf")
    y2, r2 = run(w, "silu")
    clean = torch.ones(50, 3, dtype=torch.bool, device=DEV)
    clean[20, 1] = clean[30, 2] = False
    assert torch.equal(y[clean], y2[clean]) and torch.equal(r["dx"][clean], r2["dx"][clean])
    assert y2[20, 1].isnan().all()


def test_no_rows():
    y, r = run(make((0, 3, 64), seed=23), "silu")
    assert y.shape == (0, 3, 64)
    assert not r["dweight"].any() and not r["dresidual_scale"].any()


def test_in_place():
    w = make((30, 2, 128), seed=29)
    y, _ = run(w, "silu")
    for name in ("x", "gate"):
        d = {k: None if t is None else t.to(DEV) for k, t in w.items()}
        got = kda.gated_norm_fwd(d["x"], d["gate"], d["weight"], "silu", 1e-6, d["residual"], d["residual_scale"],
                                 out=d[name])
        assert got is d[name] and torch.equal(got, y)


def test_autograd_is_gated_norm_bwd():
    w = make((2, 9, 4, 64), seed=31)
    d = {k: t.to(DEV) for k, t in w.items()}
    names = ("x", "gate", "weight", "residual", "residual_scale")
    leaves = {n: d[n].clone().requires_grad_() for n in names}
    y = kda.gated_norm(leaves["x"], leaves["gate"], leaves["weight"], "silu", 1e-6, leaves["residual"],
                       leaves["residual_scale"])
    g = torch.autograd.grad(y, [leaves[n] for n in names], d["dy"])
    _, r = run(w, "silu")
    for a, n in zip(g, names):
        assert torch.equal(a, r["d" + n]), n


def test_graph_replays_equal_eager():
    w = make((100, 4, 128), seed=37)
    _, ref_r = run(w, "sigmoid")
    d = {k: t.to(DEV) for k, t in w.items()}
    res = {}

    def call():
        res.update(kda.gated_norm_bwd(d["x"], d["gate"], d["weight"], d["dy"], "sigmoid", 1e-6, d["residual"],
                                      d["residual_scale"]))

    g = capture(call)
    for _ in range(REPLAYS):
        for t in res.values():
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for n, t in res.items():
            assert torch.equal(t, ref_r[n]), n


@pytest.mark.parametrize("kind", ["la", "kda", "gdn"])
def test_layer_forward_backward_and_decode(kind):
    """An attention block with its skip, norm and gate: outputs and every gradient
    through both operators against the fp64 chain, then one decoded token."""
    from chunked_gated_delta_kda_amd import inputs

    H, K, V, T = 2, 64, 64, 97
    gen = torch.Generator().manual_seed(41)
    if kind != "la":
        make_w = inputs.kda_workload if kind == "kda" else inputs.gdn_workload
        d = make_w(1, T, H, K, V, seed=43).to(DEV)
        v = d["v"].clone().requires_grad_()
        if kind == "kda":
            o, _ = kda.chunk_kda(d["q"], d["k"], v, d["g"], d["beta"], d["A_log"], d["dt_bias"])
        else:
            o, _ = kda.chunk_gdn(d["q"], d["k"], v, d["g"], d["beta"])
    else:
        d = {n: torch.randn(1, T, H, K, generator=gen).to(torch.bfloat16).to(DEV) for n in "qkv"}
        v = d["v"].clone().requires_grad_()
        ld = torch.tensor([-0.5, -0.01], device=DEV)
        o, S = kda.chunk_la(d["q"], d["k"], v, ld, output_final_state=True)
    w = make((1, T, H, V), seed=47)
    p = {n: w[n].to(DEV) for n in ("gate", "weight", "residual_scale", "dy")}
    y = kda.gated_norm(o, p["gate"], p["weight"], "silu", 1e-6, v, p["residual_scale"])
    (dv,) = torch.autograd.grad(y, [v], p["dy"])
    r = ref.gated_norm(o, p["gate"], p["weight"], "silu", 1e-6, v, p["residual_scale"], p["dy"])
    yr = r["y"]
    got = y.detach().double().cpu().numpy()
    assert np.linalg.norm(got - yr) <= 2.0 ** -8 * np.linalg.norm(yr)
    assert torch.isfinite(dv.float()).all()
    if kind == "la":
        # dv: the skip's part and what reaches v through the attention, each rounded to bf16 and
        # the latter carrying its own two roundings, then their sum
        lin = ref.la_bwd(d["q"], d["k"], v, ld, K ** -0.5, torch.from_numpy(r["dx"]))
        want = lin["dv"] + r["dresidual"]
        mag = np.linalg.norm(lin["dv"]) + np.linalg.norm(r["dresidual"])
        assert np.linalg.norm(dv.double().cpu().numpy() - want) <= 4 * 2.0 ** -8 * mag
        tok = {n: torch.randn(1, H, K, generator=gen).to(torch.bfloat16).to(DEV) for n in "qkv"}
        o1, S1 = kda.la_decode(tok["q"], tok["k"], tok["v"], ld, state=S.detach())
        y1 = kda.gated_norm_fwd(o1, tok["q"], p["weight"], "silu", 1e-6, tok["v"], p["residual_scale"])
        cat = {n: torch.cat([d[n], tok[n][:, None]], 1) for n in "qkv"}
        oc, _ = ref.la_fwd(cat["q"], cat["k"], cat["v"], ld, K ** -0.5)
        yc = ref.gated_norm(torch.from_numpy(oc[:, -1]), tok["q"], p["weight"], "silu", 1e-6, tok["v"],
                            p["residual_scale"])
        # the attention's output is rounded to bf16 between the two, and the result again
        assert np.linalg.norm(y1.double().cpu().numpy() - yc) <= 3 * 2.0 ** -8 * np.linalg.norm(yc)


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_closed_gates_keep_their_tail(act):
    """sigmoid(z) is subnormal from z = -88 to -103.  There e^z and what is multiplied
    by it are multiples of 2^-149 and off by a few of them (at most four roundings and
    an ulp or two of the exponential: 8 * 2^-149 times the other factors), and the
    result is a multiple of bf16's 2^-133: half a step is 2^-134."""
    w = make((16, 2, 64), seed=59, res=False)
    w["gate"] = (-86.0 - 14.0 * torch.rand(16, 2, 64, generator=torch.Generator().manual_seed(61))).to(torch.bfloat16)
    y, r = run(w, act)
    c = {k: None if t is None else t.double() for k, t in w.items()}
    want = ref.gated_norm(c["x"], c["gate"], c["weight"], act, 1e-6, None, None, c["dy"])
    x, z, wt, dy = (c[n].numpy() for n in ("x", "gate", "weight", "dy"))
    n = np.abs(x) / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6)
    factor = 1 + np.abs(z)  # (silu's z s, and z (1 - s) in its slope)
    for name, got, others in (("y", y, n * np.abs(wt)), ("dgate", r["dgate"], np.abs(dy * wt) * n)):
        g = got.double().cpu().numpy()
        tiny = 8 * 2.0 ** -149 * others * factor + 2.0 ** -134
        bad = np.abs(g - want[name]) - 2.0 ** -8 * np.abs(want[name]) - FINE * others * factor * np.exp(z) - tiny
        assert bad.max() <= 0, (name, bad.max())
        assert np.abs(want[name]).max() > 64 * 2.0 ** -133  # not all below what is told apart


def test_open_gates_keep_their_slope():
    """sigmoid'(z) = s (1 - s), of which 1 - s is e^-z for an open gate: it is to be as
    good as s is, though s is next to one (2^-17 of the product, as everywhere here, and
    below z = 80 it is normal)."""
    w = make((16, 2, 64), seed=67, res=False)
    w["gate"] = (80.0 * torch.rand(16, 2, 64, generator=torch.Generator().manual_seed(71))).to(torch.bfloat16)
    _, r = run(w, "sigmoid")
    x, z, wt, dy = (w[n].double().numpy() for n in ("x", "gate", "weight", "dy"))
    want = dy * wt * x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-6) * np.exp(-z) / (1 + np.exp(-z)) ** 2
    g = r["dgate"].double().cpu().numpy()
    bad = np.abs(g - want) - (2.0 ** -8 + FINE) * np.abs(want) - 2.0 ** -134
    assert bad.max() <= 0, bad.max()
    assert (np.abs(g) > 0).mean() > 0.9


@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("spread,eps", [(1e25, 1e-6), (1e37, 0.0), (1e-25, 0.0), (1e-18, 1e-36), (1e-30, 1e-36)])
def test_rows_whose_squares_leave_the_range(spread, eps, res):
    """The norm is of the size of one whatever the row's: squares of 1e20 or 1e-23 have
    no place in fp32."""
    w = make((40, 2, 72), seed=53, spread=spread, res=res)
    if res:  # of the row's own size
        w["residual"] = (w["residual"].double() * spread).to(torch.bfloat16)
    check(w, "silu", eps)
