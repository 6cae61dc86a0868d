"""The fp64 reference of linear attention with a decay for each head and of the
gated norm: closed forms, continuation, and gradients against differences."""
import numpy as np
import pytest
import torch

from oracle import linear as ref


def rand(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def la_case(B=2, T=7, H=2, K=3, V=4, seed=0):
    q, k, v = rand(B, T, H, K, seed=seed), rand(B, T, H, K, seed=seed + 1), rand(B, T, H, V, seed=seed + 2)
    ld = -rand(H, seed=seed + 3).abs()
    return q, k, v, ld, rand(B, H, K, V, seed=seed + 4)


def test_no_decay_is_a_cumulative_sum():
    q, k, v, ld, _ = la_case()
    o, S = ref.la_fwd(q, k, v, torch.zeros_like(ld), 0.5)
    kv = torch.einsum("bthk,bthv->bthkv", k, v).cumsum(1)
    assert np.allclose(o, 0.5 * torch.einsum("bthkv,bthk->bthv", kv, q).numpy())
    assert np.allclose(S, kv[:, -1].numpy())


def test_closed_form_with_decay_and_state():
    q, k, v, ld, h0 = la_case(seed=10)
    o, S = ref.la_fwd(q, k, v, ld, 0.7, h0)
    T = q.shape[1]
    t = torch.arange(T, dtype=torch.float64)
    gap = t[:, None] - t[None]
    dec = torch.where(gap >= 0, torch.exp(ld[:, None, None] * gap.clamp(min=0)), 0.0)
    p = torch.einsum("bihk,bjhk->bhij", q, k) * dec
    want = torch.einsum("bhij,bjhv->bihv", p, v)
    want = want + torch.einsum("bihk,bhkv,ih->bihv", q, h0, torch.exp(ld[None] * (t + 1)[:, None]))
    assert np.allclose(o, 0.7 * want.numpy())


def test_forgetting_everything_leaves_the_last_token():
    q, k, v, ld, h0 = la_case(seed=20)
    o, S = ref.la_fwd(q, k, v, torch.full_like(ld, -float("inf")), 1.0, h0)
    assert np.allclose(o, ((q * k).sum(-1, keepdim=True) * v).numpy())
    assert np.allclose(S, torch.einsum("bhk,bhv->bhkv", k[:, -1], v[:, -1]).numpy())


def test_continuation_and_packing():
    q, k, v, ld, h0 = la_case(B=1, T=11, seed=30)
    o, S = ref.la_fwd(q, k, v, ld, 1.0, h0)
    o1, S1 = ref.la_fwd(q[:, :4], k[:, :4], v[:, :4], ld, 1.0, h0)
    o2, S2 = ref.la_fwd(q[:, 4:], k[:, 4:], v[:, 4:], ld, 1.0, torch.from_numpy(S1))
    assert np.allclose(o, np.concatenate([o1, o2], 1)) and np.allclose(S, S2)
    h = torch.cat([h0, torch.from_numpy(S1), h0])
    op, Sp = ref.la_fwd(q, k, v, ld, 1.0, h, cu=[0, 4, 11, 11])
    assert np.allclose(op, o) and np.allclose(Sp[1], S[0]) and np.allclose(Sp[2], h0[0].numpy())


def slope(f, x, d, eps=1e-5):
    return (f(x + eps * d) - f(x - eps * d)) / (2 * eps)


@pytest.mark.parametrize("name", ["q", "k", "v", "h0"])
def test_la_gradients_against_differences(name):
    q, k, v, ld, h0 = la_case(T=9, seed=40)
    a = dict(q=q, k=k, v=v, h0=h0)
    do, dfin = rand(*v.shape, seed=50).numpy(), rand(*h0.shape, seed=51).numpy()

    def loss(x):
        b = dict(a, **{name: x})
        o, S = ref.la_fwd(b["q"], b["k"], b["v"], ld, 0.6, b["h0"])
        return (o * do).sum() + (S * dfin).sum()

    r = ref.la_bwd(q, k, v, ld, 0.6, torch.from_numpy(do), h0, torch.from_numpy(dfin))
    d = rand(*a[name].shape, seed=60)
    want = slope(loss, a[name], d)
    assert abs((r["d" + name] * d.numpy()).sum() - want) <= 1e-7 * max(1.0, abs(want))


@pytest.mark.parametrize("activation", ["sigmoid", "silu"])
@pytest.mark.parametrize("gated,res", [(True, True), (True, False), (False, True)])
def test_norm_gradients_against_differences(activation, gated, res):
    T, H, D = 3, 2, 8
    a = dict(x=rand(T, H, D, seed=70), gate=rand(T, H, D, seed=71) if gated else None,
             weight=rand(D, seed=72), residual=rand(T, H, D, seed=73) if res else None,
             residual_scale=rand(H, seed=74) if res else None)
    dy = rand(T, H, D, seed=75)

    def y(b):
        return ref.gated_norm(b["x"], b["gate"], b["weight"], activation, 1e-3, b["residual"],
                              b["residual_scale"])

    r = ref.gated_norm(a["x"], a["gate"], a["weight"], activation, 1e-3, a["residual"],
                       a["residual_scale"], dy)
    assert np.allclose(r["y"], y(a))
    for n, t in a.items():
        if t is None:
            continue
        d = rand(*t.shape, seed=80)
        want = slope(lambda x: (y(dict(a, **{n: x})) * dy.numpy()).sum(), t, d)
        assert abs((r["d" + n] * d.numpy()).sum() - want) <= 1e-7 * max(1.0, abs(want)), n
