"""GPU parity of linear attention with a decay for each head (la_fwd, la_bwd,
la_decode, chunk_la) against the fp64 token recurrence.

Tolerances, from the roundings of the method.  A rounding to bf16 is off by at
most 2^-8 of the value.  An output is a sum of terms of which each carries one
such rounding inside (of P or of the state's copy), and the sum is rounded once
more: |o - ref| <= 1.02 * 2^-8 (A + |ref|), A the same sum over the terms'
absolute values (the 0.02 covers second order and the fp32 sums).  The state
is fp32: per 64-token chunk at most six accumulations and one scaling round it,
each by 2^-24, and a weight is off by about 2^-22; over the 33 chunks of the
longest case here that is below 2^-16 A element by element.  Those roundings
are independent, so as a whole (Frobenius) the state is within 2^-19: sqrt(33 *
7) * 2^-25 + 2^-22 < 2^-20.  Outputs as a whole are within 2^-7 on inputs of
random sign: the rounding inside and the one outside, 2^-8 each at most.
"""
import numpy as np
import pytest
import torch

import chunked_gated_delta_kda_amd as kda
from oracle import linear as ref
from parity_util import say
from test_gpu_graph import REPLAYS, capture

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = 2.0 ** -8 * 1.02


def make(B, T, H, K, V, seed, lens=None, lead=0, tail=0, decay="slopes", init=True):
    """Seeded inputs (on the CPU); packed when ``lens`` is given, with ``lead`` and
    ``tail`` rows outside the sequences."""
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s, dt=torch.bfloat16: torch.randn(*s, generator=gen).to(dt)  # noqa: E731
    cu = None
    if lens is not None:
        B, T = 1, lead + sum(lens) + tail
        cu = torch.tensor(np.cumsum([lead] + list(lens)), dtype=torch.int32)
    N = B if lens is None else len(lens)
    ld = {"slopes": -torch.exp2(-8.0 * torch.arange(1, H + 1, dtype=torch.float32) / H),
          "none": torch.zeros(H), "all": torch.full((H,), -float("inf")),
          "fast": torch.linspace(-300.0, -3.0, H), "slow": torch.full((H,), -1e-5)}[decay]
    return dict(q=n(B, T, H, K), k=n(B, T, H, K), v=n(B, T, H, V), do=n(B, T, H, V), ld=ld, cu=cu,
                h0=n(N, H, K, V, dt=torch.float32) if init else None, dfin=n(N, H, K, V, dt=torch.float32),
                scale=K ** -0.5)


def dev(w):
    return {k: (t.to(DEV) if isinstance(t, torch.Tensor) else t) for k, t in w.items()}


def f64(t):
    return t.detach().double().cpu().numpy()


def magnitude(w):
    """The same sums over the terms' absolute values."""
    a = {k: (t.abs() if isinstance(t, torch.Tensor) and k not in ("ld", "cu") else t) for k, t in w.items()}
    o, S = ref.la_fwd(a["q"], a["k"], a["v"], a["ld"], a["scale"], a["h0"], a["cu"])
    return o, S, ref.la_bwd(a["q"], a["k"], a["v"], a["ld"], a["scale"], a["do"], a["h0"], a["dfin"], a["cu"])


def near_bf16(name, got, want, mag, whole=True):
    got = f64(got)
    assert np.all(np.isfinite(got)), name
    bad = np.abs(got - want) - BF * (mag + np.abs(want)) - 1e-30
    rel = np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-30)
    say(f"  {name}: rel {rel:.2e}, over the bound by {bad.max() if bad.size else 0:.1e}")
    assert not bad.size or bad.max() <= 0, name
    assert not whole or rel <= 2.0 ** -7, (name, rel)


def near_state(name, got, want, mag, whole=True):
    got = f64(got)
    assert np.all(np.isfinite(got)), name
    bad = np.abs(got - want) - 2.0 ** -16 * mag - 1e-30
    rel = np.linalg.norm(got - want) / max(np.linalg.norm(want), 1e-30)
    say(f"  {name}: rel {rel:.2e}, over the bound by {bad.max() if bad.size else 0:.1e}")
    assert not bad.size or bad.max() <= 0, name
    assert not whole or rel <= 2.0 ** -19, (name, rel)


def fwd(d, **kw):
    return kda.la_fwd(d["q"], d["k"], d["v"], d["ld"], d["scale"], d["h0"], cu_seqlens=d["cu"], **kw)


def bwd(d, **kw):
    return kda.la_bwd(d["q"], d["k"], d["v"], d["ld"], d["do"], d["scale"], d["h0"], d["dfin"], d["cu"], **kw)


def check(w, whole=True, gradients=True, **kw):
    say(f"[la] {[tuple(w[n].shape) for n in 'qv']} cu {None if w['cu'] is None else w['cu'].tolist()[:12]} {kw}")
    d = dev(w)
    o, S = fwd(d, **kw)
    r = bwd(d, **kw) if gradients else None
    torch.cuda.synchronize()
    mo, mS, mr = magnitude(w)
    ro, rS = ref.la_fwd(w["q"], w["k"], w["v"], w["ld"], w["scale"], w["h0"], w["cu"])
    near_bf16("o", o, ro, mo, whole)
    near_state("state", S, rS, mS, whole)
    if gradients:
        rr = ref.la_bwd(w["q"], w["k"], w["v"], w["ld"], w["scale"], w["do"], w["h0"], w["dfin"], w["cu"])
        for n in ("dq", "dk", "dv"):
            near_bf16(n, r[n], rr[n], mr[n], whole)
        near_state("dh0", r["dh0"], rr["dh0"], mr["dh0"], whole)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 63, 64, 65, 127, 128, 129, 200])
def test_lengths(T):
    check(make(2, T, 3, 64, 64, seed=100 + T), whole=T > 16)


@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
def test_head_dimensions(K, V):
    check(make(1, 150, 5, K, V, seed=200 + K + 2 * V))


@pytest.mark.parametrize("decay", ["none", "all", "fast", "slow"])
@pytest.mark.parametrize("init", [True, False])
def test_decays(decay, init):
    check(make(1, 190, 2, 64, 128, seed=300, decay=decay, init=init))


@pytest.mark.parametrize("lens,lead,tail", [([1], 0, 0), ([64, 64], 0, 0), ([0, 5, 0, 130, 1, 0], 0, 0),
                                            ([70, 0, 3], 9, 41), ([0, 0], 3, 4), ([33] * 70, 0, 1)])
def test_packed(lens, lead, tail):
    w = make(0, 0, 2, 64, 128, seed=400, lens=lens, lead=lead, tail=tail)
    check(w, whole=sum(lens) > 100)
    d = dev(w)
    nan = torch.full_like(d["v"], float("nan"))
    o, _ = fwd(d, out=nan)
    lo, hi = lead, lead + sum(lens)
    assert not o[:, :lo].any() and not o[:, hi:].any()  # rows outside every sequence: zeros
    r = bwd(d)
    for n in ("dq", "dk", "dv"):
        assert not r[n][:, :lo].any() and not r[n][:, hi:].any(), n


@pytest.mark.parametrize("chunks", [1, 3])
def test_segments(chunks):
    check(make(2, 450, 2, 64, 128, seed=500), segment_chunks=chunks)
    check(make(0, 0, 2, 128, 64, seed=501, lens=[0, 300, 64, 1, 0, 129, 192], tail=5), segment_chunks=chunks)


def test_segments_of_many_short_sequences():
    """More sequences than the slot search looks at in one step."""
    lens = [(7 * i) % 90 for i in range(200)]
    check(make(0, 0, 1, 64, 64, seed=510, lens=lens), segment_chunks=1)


@pytest.mark.parametrize("decay", ["slow", "slopes"])
def test_long_state_keeps_its_last_bits(decay):
    """2100 tokens: the rounding of a chunk's decay must not add up."""
    w = make(1, 2100, 1, 64, 64, seed=520, decay=decay)
    check(w, gradients=False)
    check(w, gradients=False, segment_chunks=4)


def test_automatic_segments_equal_whole_sequences():
    w = make(1, 6000, 1, 128, 128, seed=530)
    assert kda.la_workspace_size(1, 6000, 1, 128, 128) > 256
    d = dev(w)
    o, S = fwd(d)
    o1, S1 = fwd(d, segment_chunks=-1)
    r, r1 = bwd(d), bwd(d, segment_chunks=-1)
    assert (S - S1).norm() <= 2.0 ** -18 * S1.norm()
    assert (r["dh0"] - r1["dh0"]).norm() <= 2.0 ** -18 * r1["dh0"].norm()
    for a, b in ((o, o1), (r["dq"], r1["dq"]), (r["dk"], r1["dk"]), (r["dv"], r1["dv"])):
        assert (a.float() - b.float()).norm() <= 2.0 ** -8 * b.float().norm()


def test_nan_stays_in_its_sequence_and_head():
    w = make(0, 0, 3, 64, 64, seed=540, lens=[40, 50, 30])
    d = dev(w)
    o, S = fwd(d)
    v = d["v"].clone()
    v[0, 60, 1] = float("nan")  # sequence 1, head 1
    o2, S2 = fwd(dict(d, v=v))
    clean = torch.ones_like(o, dtype=torch.bool)
    clean[0, 40:90, 1] = False
    assert torch.equal(o[clean], o2[clean])
    assert torch.equal(S[0], S2[0]) and torch.equal(S[2], S2[2]) and torch.equal(S[1, 0], S2[1, 0])
    assert o2[0, 60:90, 1].isnan().all()


def test_no_tokens():
    d = dev(make(2, 0, 3, 64, 64, seed=550))
    o, S = fwd(d)
    assert o.shape == (2, 0, 3, 64) and torch.equal(S, d["h0"])
    r = bwd(d)
    assert torch.equal(r["dh0"], d["dfin"])


def test_gradient_of_the_state_against_differences():
    """The final state is linear in k and in the initial state: its differences
    are exact, and the gradients of <dfin, S> have to give them."""
    w = make(1, 130, 2, 64, 64, seed=560)
    w["do"].zero_()
    d = dev(w)
    r = bwd(d)
    step = torch.zeros_like(d["k"])
    step[0, 100] = 0.5
    _, S0 = fwd(dict(d, k=torch.zeros_like(d["k"])))
    _, S1 = fwd(dict(d, k=step))
    got = (r["dk"].double() * step.double()).sum()
    want = ((S1.double() - S0.double()) * d["dfin"].double()).sum()
    # dk is rounded to bf16 twice per element (inside and at the end)
    mag = (r["dk"].double().abs() * step.double()).sum()
    assert (got - want).abs() <= 4 * BF * mag
    _, Sa = fwd(dict(d, h0=2 * d["h0"]))
    _, Sb = fwd(d)
    got = (r["dh0"].double() * d["h0"].double()).sum()
    want = ((Sa.double() - Sb.double()) * d["dfin"].double()).sum()
    mag = ((Sa.abs() + Sb.abs()).double() * d["dfin"].double().abs()).sum()
    assert (got - want).abs() <= 2.0 ** -16 * mag


@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("N,H", [(1, 1), (3, 5)])
def test_decode(N, H, K, V):
    w = make(N, 1, H, K, V, seed=600 + N)
    d = dev(w)
    o, S = kda.la_decode(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["ld"], d["scale"], d["h0"])
    ro, rS = ref.la_fwd(w["q"], w["k"], w["v"], w["ld"], w["scale"], w["h0"])
    mo, mS, _ = magnitude(w)
    # fp32 but for the output's rounding
    assert np.all(np.abs(f64(o) - ro[:, 0]) <= 2.0 ** -8 * np.abs(ro[:, 0]) + 2.0 ** -16 * mo[:, 0])
    assert np.all(np.abs(f64(S) - rS) <= 2.0 ** -21 * mS)
    o0, S0 = kda.la_decode(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["ld"], d["scale"])
    oz, Sz = kda.la_decode(d["q"][:, 0], d["k"][:, 0], d["v"][:, 0], d["ld"], d["scale"], torch.zeros_like(d["h0"]))
    assert torch.equal(o0, oz) and torch.equal(S0, Sz)


@pytest.mark.parametrize("decay", ["slopes", "slow", "all"])
def test_decode_continues_a_prompt(decay):
    """A prompt, then tokens one by one with the state in place, equal the whole."""
    w = make(2, 100, 3, 64, 128, seed=610, decay=decay)
    d = dev(w)
    _, S = kda.la_fwd(d["q"][:, :60].contiguous(), d["k"][:, :60].contiguous(), d["v"][:, :60].contiguous(), d["ld"],
                      d["scale"], d["h0"])
    outs = []
    for t in range(60, 100):
        o, S2 = kda.la_decode(*(d[n][:, t].contiguous() for n in "qkv"), d["ld"], d["scale"], S, state_out=S)
        assert S2 is S
        outs.append(o)
    ro, rS = ref.la_fwd(w["q"], w["k"], w["v"], w["ld"], w["scale"], w["h0"])
    mo, mS, _ = magnitude(w)
    near_bf16("o", torch.stack(outs, 1), ro[:, 60:], mo[:, 60:])
    near_state("state", S, rS, mS)


def test_autograd_is_la_bwd():
    d = dev(make(0, 0, 2, 64, 128, seed=620, lens=[90, 0, 40], tail=3))
    leaves = {n: d[n].clone().requires_grad_() for n in ("q", "k", "v", "h0")}
    o, S = kda.chunk_la(leaves["q"], leaves["k"], leaves["v"], d["ld"], d["scale"], leaves["h0"], True, d["cu"])
    g = torch.autograd.grad([o, S], list(leaves.values()), [d["do"], d["dfin"]])
    r = bwd(d)
    for a, n in zip(g, ("dq", "dk", "dv", "dh0")):
        assert torch.equal(a, r[n]), n
    # the output alone, with a gradient that is no dense tensor
    o, none = kda.chunk_la(leaves["q"], leaves["k"], leaves["v"], d["ld"], d["scale"], None, False, d["cu"])
    assert none is None
    (gq,) = torch.autograd.grad(o.sum(), [leaves["q"]])
    r = kda.la_bwd(d["q"], d["k"], d["v"], d["ld"], torch.ones_like(o), d["scale"], cu_seqlens=d["cu"])
    assert torch.equal(gq, r["dq"])


@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("T", [64, 130, 448])
def test_same_results_every_time(K, V, T):
    """No result depends on when a wave gets there."""
    d = dev(make(4, T, 8, K, V, seed=625))
    o, S = fwd(d)
    r = bwd(d)
    for _ in range(20):
        o2, S2 = fwd(d)
        r2 = bwd(d)
        assert torch.equal(o, o2) and torch.equal(S, S2)
        for n in r:
            assert torch.equal(r[n], r2[n]), n


def test_same_results_twice_and_on_another_stream():
    d = dev(make(1, 700, 3, 128, 128, seed=630))
    o, S = fwd(d, segment_chunks=2)
    r = bwd(d, segment_chunks=2)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        o2, S2 = fwd(d, segment_chunks=2)
        r2 = bwd(d, segment_chunks=2)
    s.synchronize()
    assert torch.equal(o, o2) and torch.equal(S, S2)
    for n in r:
        assert torch.equal(r[n], r2[n]), n


def test_graph_replays_equal_eager():
    w = make(0, 0, 2, 64, 64, seed=640, lens=[150, 1, 80])
    d = dev(w)
    ws = torch.empty(kda.la_workspace_size(1, w["q"].shape[1], 2, 64, 64, 3, 1, backward=True), dtype=torch.uint8,
                     device=DEV)
    out, fin = torch.empty_like(d["v"]), torch.empty_like(d["h0"])
    res = {}

    def call():
        fwd(d, workspace=ws, out=out, final_out=fin, segment_chunks=1)
        res.update(bwd(d, workspace=ws, segment_chunks=1))

    call()
    torch.cuda.synchronize()
    want = {n: t.clone() for n, t in dict(res, out=out, fin=fin).items()}
    g = capture(call)
    got = dict(res, out=out, fin=fin)
    for rep in range(REPLAYS):
        for t in got.values():
            t.fill_(float("nan"))
        ws.fill_(255)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for n, t in got.items():
            assert torch.equal(t, want[n]), (rep, n)


def test_rows_past_32_bit_offsets():
    """A batch of 3.2 billion elements a tensor: its last sequence equals the same
    tokens alone."""
    H, T, last = 96, 262144, 150
    gen = torch.Generator(device=DEV).manual_seed(650)
    big = {n: torch.empty(1, T, H, 128, dtype=torch.bfloat16, device=DEV) for n in ("q", "k", "v", "do")}
    for t in big.values():
        t[:, :64].normal_(generator=gen)
        t[:, 64:-last].zero_()
        t[:, -last:].normal_(generator=gen)
    ld = torch.full((H,), -0.05, device=DEV)
    cu = torch.tensor([0, T - last, T], dtype=torch.int32, device=DEV)
    o, S = kda.la_fwd(big["q"], big["k"], big["v"], ld, cu_seqlens=cu)
    tail = {n: t[:, -last:].contiguous() for n, t in big.items()}
    o1, S1 = kda.la_fwd(tail["q"], tail["k"], tail["v"], ld)
    assert torch.equal(o[:, -last:], o1) and torch.equal(S[1], S1[0])
    del o
    r = kda.la_bwd(big["q"], big["k"], big["v"], ld, big["do"], cu_seqlens=cu)
    r1 = kda.la_bwd(tail["q"], tail["k"], tail["v"], ld, tail["do"])
    for n in ("dq", "dk", "dv"):
        assert torch.equal(r[n][:, -last:], r1[n]), n
    assert torch.equal(r["dh0"][1], r1["dh0"][0])


# more (sequence, head) pairs than one round of narrow workgroups holds
MANY = 130


@pytest.mark.parametrize("K,V", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("T", [1, 64, 100, 193])
def test_many_heads(T, K, V):
    check(make(1, T, 2 * MANY if V == 64 else MANY, K, V, seed=700 + T + K + 2 * V), whole=T > 16)


@pytest.mark.parametrize("decay", ["none", "all", "fast", "slow"])
def test_many_heads_decays(decay):
    check(make(1, 150, MANY, 128, 128, seed=710, decay=decay), gradients=True)


@pytest.mark.parametrize("lens,lead,tail", [([0, 5, 0, 130, 1, 0], 0, 0), ([70, 0, 3], 9, 41), ([33] * 63, 0, 1),
                                            ([33, 7, 90] * 22, 2, 0)])
def test_many_heads_packed(lens, lead, tail):
    """Longest first up to 64 sequences, in order beyond."""
    w = make(0, 0, 90, 64, 128, seed=720, lens=lens, lead=lead, tail=tail)
    check(w, whole=sum(lens) > 100)
    d = dev(w)
    o, _ = fwd(d, out=torch.full_like(d["v"], float("nan")))
    assert not o[:, :lead].any() and not o[:, lead + sum(lens):].any()


def test_a_head_is_the_same_beside_few_and_many():
    w = make(2, 300, MANY, 128, 128, seed=730)
    d = dev(w)
    o, S = fwd(d)
    r = bwd(d)
    one = {n: (t[:, :, 7:8].contiguous() if n in ("q", "k", "v", "do") else t) for n, t in d.items()}
    one.update(ld=d["ld"][7:8].contiguous(), h0=d["h0"][:, 7:8].contiguous(), dfin=d["dfin"][:, 7:8].contiguous())
    o1, S1 = fwd(one, segment_chunks=-1)
    r1 = bwd(one, segment_chunks=-1)
    assert torch.equal(o[:, :, 7:8], o1) and torch.equal(S[:, 7:8], S1)
    for n in ("dq", "dk", "dv"):
        assert torch.equal(r[n][:, :, 7:8], r1[n]), n
    assert torch.equal(r["dh0"][:, 7:8], r1["dh0"])


def test_gradients_without_the_states():
    """Nobody reads the last state: two terms of a decayed value are enough then."""
    w = make(1, 190, MANY, 128, 128, seed=740)
    d = dev(w)
    r = kda.la_bwd(d["q"], d["k"], d["v"], d["ld"], d["do"], d["scale"], d["h0"], d["dfin"], need_dh0=False)
    assert r["dh0"] is None
    rr = ref.la_bwd(w["q"], w["k"], w["v"], w["ld"], w["scale"], w["do"], w["h0"], w["dfin"], None)
    mr = magnitude(w)[2]
    for n in ("dq", "dk", "dv"):
        # (what two terms of eight bits cut off is below 2^-14 of the value: inside the
        # bound's 0.02 * 2^-8, beside 2^-16 for the second order)
        near_bf16(n, r[n], rr[n], mr[n])


def test_long_state_of_many_heads_keeps_its_last_bits():
    w = make(1, 2100, MANY, 64, 64, seed=750, decay="slow")
    d = dev(w)
    assert kda.la_workspace_size(1, 2100, 2 * MANY, 64, 64) <= 256
    o, S = kda.la_fwd(*(torch.cat([d[n]] * 2, 2) for n in ("q", "k", "v")), torch.cat([d["ld"]] * 2), d["scale"],
                      torch.cat([d["h0"]] * 2, 1))
    ro, rS = ref.la_fwd(*(w[n][:, :, :3] for n in ("q", "k", "v")), w["ld"][:3], w["scale"], w["h0"][:, :3], None)
    a = {n: w[n][:, :, :3].abs() for n in ("q", "k", "v")}
    mo, mS = ref.la_fwd(a["q"], a["k"], a["v"], w["ld"][:3], w["scale"], w["h0"][:, :3].abs(), None)
    near_bf16("o", o[:, :, :3], ro, mo)
    near_state("state", S[:, :3], rS, mS)
    assert torch.equal(S[:, :MANY], S[:, MANY:]) and torch.equal(o[:, :, :MANY], o[:, :, MANY:])


@pytest.mark.parametrize("K,V", [(64, 128), (128, 64), (64, 64), (128, 128)])
@pytest.mark.parametrize("H", [2, MANY])
def test_outputs_without_the_last_state(H, K, V):
    w = make(1, 130, H, K, V, seed=760)
    d = dev(w)
    o, S = kda.la_fwd(d["q"], d["k"], d["v"], d["ld"], d["scale"], d["h0"], output_final_state=False)
    assert S is None
    near_bf16("o", o, ref.la_fwd(w["q"], w["k"], w["v"], w["ld"], w["scale"], w["h0"])[0], magnitude(w)[0])


def test_no_second_derivative():
    d = dev(make(1, 70, 2, 64, 64, seed=770))
    leaf = {n: d[n].clone().requires_grad_() for n in ("q", "k", "v")}
    o, _ = kda.chunk_la(leaf["q"], leaf["k"], leaf["v"], d["ld"])
    y = kda.gated_norm(o, leaf["v"], torch.ones(64, device=DEV))
    (g,) = torch.autograd.grad(y.float().square().sum(), leaf["q"], create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable|does not require grad"):
        g.float().sum().backward()


def test_workspaces_that_are_not_one_piece_are_refused():
    d = dev(make(1, 300, 2, 64, 64, seed=780))
    size = kda.la_workspace_size(1, 300, 2, 64, 64, segment_chunks=1, backward=True)
    for ws in (torch.empty(1, dtype=torch.uint8, device=DEV).expand(size),
               torch.empty(2 * size, dtype=torch.uint8, device=DEV)[::2]):
        for call in (fwd, bwd):
            with pytest.raises(ValueError, match="contiguous"):
                call(d, workspace=ws, segment_chunks=1)
        with pytest.raises(ValueError, match="contiguous"):
            kda.gated_norm_bwd(d["q"], None, torch.ones(64, device=DEV), d["do"], workspace=ws)


def test_automatic_segments_of_a_packed_batch():
    lens, H = [9000, 1, 0, 13000, 64], 2
    T = sum(lens) + 11
    for backward in (False, True):
        assert kda.la_workspace_size(1, T, H, 128, 64, len(lens), backward=backward) > 256
    d = dev(make(0, 0, H, 128, 64, seed=790, lens=lens, lead=4, tail=7))
    o, S = fwd(d)
    o1, S1 = fwd(d, segment_chunks=-1)
    r, r1 = bwd(d), bwd(d, segment_chunks=-1)
    assert (S - S1).norm() <= 2.0 ** -18 * S1.norm()
    assert (r["dh0"] - r1["dh0"]).norm() <= 2.0 ** -18 * r1["dh0"].norm()
    for a, b in ((o, o1), (r["dq"], r1["dq"]), (r["dk"], r1["dk"]), (r["dv"], r1["dv"])):
        assert (a.float() - b.float()).norm() <= 2.0 ** -8 * b.float().norm()
        assert not a[:, :4].any() and not a[:, -7:].any()


@pytest.mark.parametrize("H", [3, MANY])
def test_outputs_carry_two_roundings(H):
    """On inputs of random sign a rounding to bf16 is off by u = 2^-8 / sqrt(3) *
    sqrt(3 / (8 ln 2)) = 1.66e-3 of the value as a root mean square (uniform in half a
    step of 2^-8, over a mantissa spread evenly over its logarithm).  Terms with one
    such rounding each, added up with random signs and rounded again, are off by
    sqrt(2) u = 2.35e-3 as a whole; a tenth more is for the sample."""
    w = make(1, 333, H, 64, 128, seed=800)
    d = dev(w)
    o, _ = fwd(d)
    r = bwd(d)
    one = {n: (t[:, :, :3] if n in ("q", "k", "v", "do") else t) for n, t in w.items()}
    one.update(ld=w["ld"][:3], h0=w["h0"][:, :3], dfin=w["dfin"][:, :3])
    want = dict(ref.la_bwd(one["q"], one["k"], one["v"], one["ld"], w["scale"], one["do"], one["h0"], one["dfin"]),
                o=ref.la_fwd(one["q"], one["k"], one["v"], one["ld"], w["scale"], one["h0"])[0])
    for n, got in dict(r, o=o).items():
        if n == "dh0":
            continue
        rel = np.linalg.norm(f64(got[:, :, :3]) - want[n]) / np.linalg.norm(want[n])
        say(f"  {n}: rel {rel:.2e}")
        assert rel <= 1.1 * 2 ** 0.5 * 1.66e-3, n
