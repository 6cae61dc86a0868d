"""GPU parity of the gated linear recurrence (gated_scan_fwd, gated_scan_bwd,
gated_scan_decode, gated_scan) against the fp64 recurrence.

Tolerances: one rounding to the tokens' type, and the bound that the reference
carries along the recurrence (2^-20 of each step's absolute terms)."""
import pytest
import torch

import chunked_gated_delta_kda_amd as kda
from block_util import DEV, TYPES, near, offsets, to_gpu
from oracle import block as ref
from parity_util import say
from test_gpu_graph import REPLAYS, capture

pytestmark = pytest.mark.gpu


def make(B, T, C, seed, dtype="bf16", init=True, cu=None, slow=-4.0, spread=1.0):
    """Decays from a few tokens to about a thousand (slow: the mean of dt_bias)."""
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    N = B if cu is None else len(cu) - 1
    tt = TYPES[dtype]
    return dict(x=(n(B, T, C) * spread).to(tt), g=n(B, T, C).to(tt), gate=(2 * n(B, T, C)).to(tt),
                A_log=n(C), dt_bias=2 * n(C) + slow, h0=n(N, C) if init else None, cu=cu,
                do=n(B, T, C).to(tt), dfinal=n(N, C))


def args(d):
    return d["x"], d["g"], d["gate"], d["A_log"], d["dt_bias"]


def run(w, **kw):
    d = to_gpu(w)
    o, f, states = kda.gated_scan_fwd_save(*args(d), d["h0"], cu_seqlens=d["cu"], **kw)
    r = kda.gated_scan_bwd(*args(d), d["do"], states, d["h0"], d["dfinal"], d["cu"])
    return o, f, r


def check(w):
    o, f, r = run(w)
    torch.cuda.synchronize()
    say(f"[scan] {tuple(w['x'].shape)} {w['x'].dtype} init {w['h0'] is not None} packed {w['cu'] is not None}")
    want = ref.scan_all(*args(w), w["h0"], w["cu"], w["do"], w["dfinal"])
    near("o", o, want["o"])
    near("final", f, want["final"])
    for got, name in (("dx", "x"), ("dg", "g"), ("dinput_gate", "i"), ("dA_log", "A_log"), ("ddt_bias", "dt_bias"),
                      ("dh0", "h0")):
        near(got, r[got], want[name])
    return o, f, r


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 64, 65, 127, 128, 129, 192, 255, 256, 257, 300])
def test_lengths(T, dtype):
    check(make(2, T, 24, seed=T, dtype=dtype))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("C", [8, 56, 64, 72, 128, 136, 360])
def test_channels(C, dtype):
    check(make(1, 37, C, seed=C, dtype=dtype))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("init", [True, False])
def test_long(init, dtype):
    check(make(2, 1500, 136, seed=3, dtype=dtype, init=init, slow=-7.0))


LENS = [[5], [0, 5, 0], [1, 1, 1, 14, 130], [16, 112, 128, 1, 0, 0, 3], [300, 0, 17], [0, 0], [1] * 40]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("tail", [0, 21, 150])
@pytest.mark.parametrize("lens", LENS)
def test_packed(lens, tail, dtype):
    cu = offsets(lens)
    T = int(cu[-1]) + tail
    if T == 0:
        pytest.skip("no rows: test_no_tokens")
    w = make(1, T, 72, seed=len(lens), dtype=dtype, cu=cu)
    for n in ("x", "g", "gate", "do"):  # rows outside count for nothing, whatever they hold
        w[n][:, int(cu[-1]):] = float("nan")
    o, _, r = check(w)
    for t in (o, r["dx"], r["dg"], r["dinput_gate"]):
        assert not t[:, int(cu[-1]):].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", [[700], [16, 112, 128, 1, 0, 300, 3, 77], [1] * 150 + [250]])
def test_packed_in_many_chains(lens, dtype):
    """More than ten chains: a tile waits for the eighth before it."""
    cu = offsets(lens)
    w = make(1, int(cu[-1]) + 5, 712, seed=len(lens), dtype=dtype, cu=cu)
    for n in ("x", "g", "gate", "do"):
        w[n][:, int(cu[-1]):] = float("nan")
    o, f, r = check(w)
    d = to_gpu(w)
    cut = slice(640, 712)
    part = [t[..., cut].contiguous() for t in args(d)]
    o1, f1, s1 = kda.gated_scan_fwd_save(*part, d["h0"][:, cut].contiguous(), cu_seqlens=d["cu"])
    r1 = kda.gated_scan_bwd(*part, d["do"][..., cut].contiguous(), s1, d["h0"][:, cut].contiguous(),
                            d["dfinal"][:, cut].contiguous(), d["cu"])
    assert torch.equal(o[..., cut], o1) and torch.equal(f[:, cut], f1)
    for k, v in r1.items():
        assert torch.equal(r[k][..., cut], v), k


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_long_in_many_chains(dtype):
    check(make(3, 1500, 264, seed=5, dtype=dtype, slow=-7.0))


def test_packed_that_begins_late():
    """Rows in front of the first sequence are outside every one, too."""
    cu = torch.tensor([20, 150, 150, 290], dtype=torch.int32)
    w = make(1, 300, 64, seed=11, cu=cu)
    o, _, r = check(w)
    assert not o[:, :20].any() and not r["dx"][:, :20].any() and not o[:, 290:].any()


def test_packed_is_each_sequence_by_itself():
    lens = [200, 1, 77, 128, 256, 5]
    cu = offsets(lens)
    w = make(1, int(cu[-1]), 128, seed=13, cu=cu, init=True)
    d = to_gpu(w)
    o, f = kda.gated_scan_fwd(*args(d), d["h0"], cu_seqlens=d["cu"])
    for n, (a, e) in enumerate(zip(cu[:-1].tolist(), cu[1:].tolist())):
        part = [d[k][:, a:e].contiguous() for k in ("x", "g", "gate")]
        o1, f1 = kda.gated_scan_fwd(*part, d["A_log"], d["dt_bias"], d["h0"][n:n + 1].contiguous())
        # tiles cut a sequence elsewhere: fp32 rounding, then one of the outputs
        assert (o[:, a:e].float() - o1.float()).abs().max() <= 2.0 ** -7 * o1.float().abs().max()
        assert (f[n] - f1[0]).abs().max() <= 2.0 ** -16 * f1.abs().max()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gates_at_the_ends(dtype):
    """Decays that are one or zero, inputs that are shut or open."""
    w = make(1, 40, 64, seed=17, dtype=dtype)
    w["dt_bias"][:8] = -200.0   # no decay at all: the state stays, and nothing enters
    w["dt_bias"][8:16] = -30.0  # a decay that 1 - a would lose
    w["dt_bias"][16:24] = 200.0  # everything is forgotten at once
    w["A_log"][16:24] = 3.0
    w["gate"][..., 24:32] = -300.0
    w["gate"][..., 32:40] = 300.0
    o, f, r = run(w)
    want = ref.scan_all(*args(w), w["h0"], None, w["do"], w["dfinal"])
    # e^-|z| is off by |z| 2^-24 of itself: for |z| up to 33, 2^-19, where the others have 2^-20
    loose = lambda n: (want[n][0], 4 * want[n][1])  # noqa: E731
    near("o", o, loose("o"))
    near("final", f, loose("final"))
    keep = [c for c in range(64) if not c < 8]
    for got, name in (("dx", "x"), ("dinput_gate", "i"), ("dh0", "h0"), ("dg", "g"), ("dA_log", "A_log"),
                      ("ddt_bias", "dt_bias")):
        v, b = loose(name)
        near(got, r[got][..., keep], (v[..., keep], b[..., keep]))
        assert torch.isfinite(r[got].float()).all(), got
    assert torch.equal(f[0, :8].cpu(), w["h0"][0, :8])
    assert not r["dx"][..., :8].any() and not r["dg"][..., :8].any()


def test_nan_stays_in_its_channel_and_sequence():
    lens = [150, 40, 300]
    cu = offsets(lens)
    w = make(1, 490, 72, seed=19, cu=cu)
    o, f, r = run(w)
    w["x"][0, 160, 5] = float("nan")
    w["g"][0, 165, 9] = float("nan")
    w["gate"][0, 3, 11] = float("inf")
    w["x"][0, 170, 20] = float("inf")
    w["do"][0, 170, 30] = float("nan")
    o2, f2, r2 = run(w)
    clean = torch.ones(490, 72, dtype=torch.bool, device=DEV)
    for c in (5, 9, 20, 30):
        clean[150:190, c] = False
    clean[:150, 11] = False
    for a, b in ((o, o2), (r["dx"], r2["dx"]), (r["dg"], r2["dg"]), (r["dinput_gate"], r2["dinput_gate"])):
        assert torch.equal(a[0][clean], b[0][clean])
    assert o2[0, 160:190, 5].isnan().all() and not o2[0, 150:160, 5].isnan().any()
    ok = torch.ones(72, dtype=torch.bool, device=DEV)
    ok[[5, 9, 11, 20, 30]] = False
    assert torch.equal(r["dA_log"][ok], r2["dA_log"][ok]) and torch.equal(f[:, ok], f2[:, ok])
    assert torch.equal(f[2], f2[2])


@pytest.mark.parametrize("C", [72, 712])  # (few chains and many)
@pytest.mark.parametrize("packed", [False, True])
def test_nan_reaches_its_sequences_end_however_fast_it_forgets(packed, C):
    """Decays whose products underflow within a tile, or that are zero: a NaN goes on all the
    same, forward in the state and backward in its gradient."""
    cu = offsets([40, 900, 70]) if packed else None
    w = make(1, 1010, C, seed=23, cu=cu)
    w["dt_bias"][:4] = 5.0
    w["A_log"][:2] = 0.0
    w["A_log"][2:4] = 5.0  # (exp(-148 L): zero)
    clean = run(w)[0]
    w["x"][0, 50, :4] = float("nan")
    w["do"][0, 930, 8] = float("nan")
    w["dt_bias"][8] = 40.0
    o, f, r = run(w)
    end = 940 if packed else 1010
    assert o[0, 50:end, :4].isnan().all() and not o[0, :50, :4].isnan().any()
    assert f[1 if packed else 0, :4].isnan().all()
    first = 40 if packed else 0
    assert r["dx"][0, first:931, 8].isnan().all() and not r["dx"][0, 931:, 8].isnan().any()
    assert not r["dx"][0, :first, 8].isnan().any() and not o[0, end:].isnan().any()
    assert torch.equal(o[..., 16:], clean[..., 16:])


@pytest.mark.parametrize("packed", [False, True])
def test_no_tokens(packed):
    cu = torch.zeros(4, dtype=torch.int32) if packed else None
    w = make(1 if packed else 3, 0, 16, seed=23, cu=cu)
    o, f, r = run(w)
    assert o.numel() == 0 and torch.equal(f.cpu(), w["h0"]) and torch.equal(r["dh0"].cpu(), w["dfinal"])
    assert not r["dA_log"].any() and not r["ddt_bias"].any()
    w["h0"] = None
    assert not run(w)[1].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("N,C", [(1, 8), (3, 360), (64, 4096)])
def test_decode_continues_the_forward_pass(N, C, dtype):
    w = make(N, 9, C, seed=C, dtype=dtype)
    d = to_gpu(w)
    want = ref.scan_all(*args(w), w["h0"])
    part = [d[k][:, :8].contiguous() for k in ("x", "g", "gate")]
    _, state = kda.gated_scan_fwd(*part, d["A_log"], d["dt_bias"], d["h0"])
    tok = [d[k][:, 8].contiguous() for k in ("x", "g", "gate")]
    before = state.clone()
    o, new = kda.gated_scan_decode(*tok, d["A_log"], d["dt_bias"], state=state)
    near("o", o, tuple(t[:, 8] for t in want["o"]))
    near("state", new, want["final"])
    assert torch.equal(state, before)
    o2, new2 = kda.gated_scan_decode(*tok, d["A_log"], d["dt_bias"], state=state, state_out=state)
    assert new2 is state and torch.equal(o, o2) and torch.equal(state, new)
    o3, new3 = kda.gated_scan_decode(*tok, d["A_log"], d["dt_bias"])
    o4, new4 = kda.gated_scan_decode(*tok, d["A_log"], d["dt_bias"], state=torch.zeros_like(new))
    assert torch.equal(o3, o4) and torch.equal(new3, new4)


def test_equal_calls_give_equal_bits():
    w = make(2, 3000, 256, seed=29)
    d = to_gpu(w)
    ws = torch.empty(kda.gated_scan_workspace_size(2, 3000, 256, True), dtype=torch.uint8, device=DEV)
    first = None
    for fill in (0, 255, 127):
        ws.fill_(fill)  # (what a workspace holds does not matter)
        o, f, s = kda.gated_scan_fwd_save(*args(d), d["h0"], workspace=ws)
        ws.fill_(fill)
        r = kda.gated_scan_bwd(*args(d), d["do"], s, d["h0"], d["dfinal"], workspace=ws)
        now = [o, f, s] + list(r.values())
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))
    o, f = kda.gated_scan_fwd(*args(d), d["h0"])
    assert torch.equal(o, first[0]) and torch.equal(f, first[1])


def test_autograd_is_gated_scan_bwd():
    cu = offsets([70, 0, 30])
    w = make(1, 100, 64, seed=31, cu=cu)
    d = to_gpu(w)
    names = ("x", "g", "gate", "A_log", "dt_bias", "h0")
    lv = {n: d[n].clone().requires_grad_() for n in names}
    o, f = kda.gated_scan(*args(lv), lv["h0"], True, d["cu"])
    got = torch.autograd.grad([o, f], list(lv.values()), [d["do"], d["dfinal"]])
    _, _, r = run(w)
    for a, n in zip(got, ("dx", "dg", "dinput_gate", "dA_log", "ddt_bias", "dh0")):
        assert torch.equal(a, r[n]), n
    # one of the outputs alone
    (gx,) = torch.autograd.grad(kda.gated_scan(*args(lv), lv["h0"], True, d["cu"])[1], [lv["x"]], d["dfinal"])
    d["do"] = torch.zeros_like(d["do"])
    assert torch.equal(gx, run({**w, "do": torch.zeros_like(w["do"])})[2]["dx"])


def test_gradients_against_differences():
    """The forward kernel's own differences, in a direction of each input."""
    w = make(1, 150, 16, seed=37, dtype="fp32", slow=-2.0)
    d = to_gpu(w)
    _, _, r = run(w)
    gen = torch.Generator().manual_seed(38)

    def loss(v):
        o, f = kda.gated_scan_fwd(*args(v), v["h0"])
        return (o.double() * d["do"].double()).sum() + (f.double() * d["dfinal"].double()).sum()

    for n, gname in (("x", "dx"), ("g", "dg"), ("gate", "dinput_gate"), ("A_log", "dA_log"), ("dt_bias", "ddt_bias"),
                     ("h0", "dh0")):
        way = torch.randn(d[n].shape, generator=gen).to(DEV)
        eps = 2.0 ** -8
        up, down = loss({**d, n: d[n] + eps * way}), loss({**d, n: d[n] - eps * way})
        want = (r[gname].double() * way.double()).sum()
        # third derivatives: eps^2 of terms of the gradient's size; roundings of o: 2^-20 / eps
        size = (r[gname].double() * way.double()).norm() + 1.0
        assert ((up - down) / (2 * eps) - want).abs() <= 2.0 ** -8 * size, n


def test_graphs_that_share_a_workspace():
    w = make(1, 700, 128, seed=41)
    d = to_gpu(w)
    v = {k: t.flip(1).contiguous() if k in ("x", "g", "gate", "do") else t for k, t in d.items() if t is not None}
    ws = torch.empty(kda.gated_scan_workspace_size(1, 700, 128, True), dtype=torch.uint8, device=DEV)

    def both(q, out):
        o, f, s = kda.gated_scan_fwd_save(*args(q), q["h0"], workspace=ws)
        r = kda.gated_scan_bwd(*args(q), q["do"], s, q["h0"], q["dfinal"], workspace=ws)
        out[:] = [o, f] + list(r.values())

    want, res, graphs = [], [], []
    for q in (d, v):
        out = []
        both(q, out)
        want.append([t.clone() for t in out])
        keep = []
        graphs.append(capture(lambda q=q, keep=keep: both(q, keep)))
        res.append(keep)
    for k in range(2 * REPLAYS):
        i = k % 2
        for t in res[i]:
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(res[i], want[i])), k


def test_two_streams_at_once():
    ws = [make(1, 2000, 256, seed=s) for s in (43, 44)]
    want = [run(w) for w in ws]
    d = [to_gpu(w) for w in ws]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ws]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(kda.gated_scan_fwd(*args(d[i]), d[i]["h0"]))
    torch.cuda.synchronize()
    for i in range(2):
        for o, f in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(f, want[i][1])


def test_large_values_in_the_last_row():
    """Rows behind the last token are read as the last one, without a decay: nothing of
    them, however large, reaches the sums over tokens."""
    w = make(2, 70, 24, seed=47, dtype="fp32")
    w["x"][:, -1] *= 2.0 ** 90
    check(w)


@pytest.mark.parametrize("B,T", [(11, 260), (1, 4300), (300, 4000), (16, 1400)])
def test_counters_and_looks(B, T):
    """Tiles in 33 chains, one, 300 or 16: where they are more than ten a tile looks at 8
    before it, not at 32, and finds the same sums in the same order."""
    C = 136 if B == 11 else 64
    gen = torch.Generator(device=DEV).manual_seed(B)
    n = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    x, g, i, do = (n(B, T, C) for _ in range(4))
    A, bias, h0, df = n(C), 2 * n(C) - 5, n(B, C), n(B, C)
    o, f, s = kda.gated_scan_fwd_save(x, g, i, A, bias, h0)
    r = kda.gated_scan_bwd(x, g, i, A, bias, do, s, h0, df)
    for b in sorted({0, B // 2, B - 1}):
        one = [t[b:b + 1].contiguous() for t in (x, g, i, do, h0, df)]
        o1, f1, s1 = kda.gated_scan_fwd_save(*one[:3], A, bias, one[4])
        r1 = kda.gated_scan_bwd(*one[:3], A, bias, one[3], s1, one[4], one[5])
        assert torch.equal(o[b], o1[0]) and torch.equal(f[b], f1[0])
        for k in ("dx", "dg", "dinput_gate", "dh0"):
            assert torch.equal(r[k][b], r1[k][0]), k
