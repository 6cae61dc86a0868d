"""The operators around a block one behind the other, as a block runs them: trained
against the fp64 chain, and token by token behind a prompt; in front of and behind KDA
attention; and what their wrappers refuse on a GPU."""
import pytest
import torch

import chunked_gated_delta_kda_amd as kda
from block_util import DEV, TYPES
from chunked_gated_delta_kda_amd import inputs
from oracle import block as ref

pytestmark = pytest.mark.gpu

# The chain rounds eleven times to the tokens' type (u, y, c, o, u', y' and five gradients
# between them), each time by half a step of each element; norms, taps whose squares add
# up to one and a recurrence that only forgets hand on at most twice what they get.  fp32's
# arithmetic is counted as 2^-20 (see oracle/block.py) for each of them, and four times that
# in a recurrence whose decays stay below 3/4.
TOL = {"bf16": 11 * 2 * 2.0 ** -8, "fp32": 11 * 2 * 4 * 2.0 ** -20}


def make(B, T, C, dtype, seed, W=4):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    tt = TYPES[dtype]
    tokens = {k: n(B, T, C).to(tt) for k in ("x", "res", "g", "gate", "way")}
    tokens["g"] = (tokens["g"] / 4).clamp(-1, 1)
    return dict(tokens, w1=1 + n(C) / 8, b1=n(C) / 8, taps=n(C, W) / 2, cb=n(C) / 8, A_log=n(C) / 8,
                dt_bias=0.5 + n(C).clamp(-1, 1) / 4, w2=1 + n(C) / 8, b2=n(C) / 8)


LEAVES = ("x", "res", "g", "gate", "w1", "b1", "taps", "cb", "A_log", "dt_bias", "w2", "b2")


def block(d, cu=None):
    y, u = kda.layer_norm(d["x"], d["w1"], d["b1"], residual=d["res"])
    c, cs = kda.short_conv(y, d["taps"], d["cb"], output_final_state=True, cu_seqlens=cu)
    o, hs = kda.gated_scan(c, d["g"], d["gate"], d["A_log"], d["dt_bias"], output_final_state=True, cu_seqlens=cu)
    out, _ = kda.layer_norm(o, d["w2"], d["b2"], residual=u)
    return out, cs, hs


def block64(d, cu=None):
    u = d["x"] + d["res"]
    c, _, _ = ref.conv(ref.layer_norm(u, d["w1"], d["b1"]), d["taps"], d["cb"], "silu", None, cu)
    o, hs = ref.scan(c, d["g"], d["gate"], d["A_log"], d["dt_bias"], None, cu)
    return ref.layer_norm(o + u, d["w2"], d["b2"]), hs


def off(a, b):
    return ((a.detach().double().cpu() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens", [None, [70, 0, 1, 133, 3]])
def test_a_block_is_trained(lens, dtype):
    cu = None if lens is None else torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32)
    w = make(*((2, 150) if lens is None else (1, int(cu[-1]))), 72, dtype, seed=61)
    d = {k: t.to(DEV).requires_grad_(k in LEAVES) for k, t in w.items()}
    out, _, hs = block(d, None if cu is None else cu.to(DEV))
    (out * d["way"]).sum().backward()
    q = {k: t.double().requires_grad_(k in LEAVES) for k, t in w.items()}
    want, hs64 = block64(q, cu)
    (want * q["way"]).sum().backward()
    assert off(out, want.detach()) <= TOL[dtype] and off(hs, hs64.detach()) <= TOL[dtype]
    for n in LEAVES:
        assert d[n].grad.dtype == d[n].dtype and off(d[n].grad, q[n].grad) <= TOL[dtype], n


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_prompt_and_the_tokens_behind_it(dtype):
    B, T, more = 3, 140, 6
    w = make(B, T + more, 64, dtype, seed=67)
    d = {k: t.to(DEV) for k, t in w.items()}
    front = {k: t[:, :T].contiguous() if t.dim() == 3 else t for k, t in d.items()}
    out, cs, hs = block(front)
    got = [out]
    for t in range(T, T + more):
        x, r, g, i = (d[k][:, t].contiguous() for k in ("x", "res", "g", "gate"))
        y, u = kda.layer_norm_fwd(x, d["w1"], d["b1"], residual=r)
        c, _ = kda.short_conv_decode(y, d["taps"], cs, d["cb"], state_out=cs)
        o, _ = kda.gated_scan_decode(c, g, i, d["A_log"], d["dt_bias"], hs, state_out=hs)
        out, _ = kda.layer_norm_fwd(o, d["w2"], d["b2"], residual=u)
        got.append(out[:, None])
    got = torch.cat(got, 1)
    want, hs64 = block64({k: t.double() for k, t in w.items()})
    for t in list(range(T, T + more)) + [0, T - 1]:
        assert off(got[:, t], want[:, t]) <= TOL[dtype], t
    assert off(hs, hs64) <= TOL[dtype]


def test_convolutions_in_front_of_kda_and_the_norm_behind_it():
    """q, k and v as a layer has them; autograd hands the kernels' own gradients on."""
    B, T, H, D = 2, 90, 2, 64
    w = inputs.kda_workload(B, T, H, D, D, seed=71, dt_bias_value=-6.0, init_std=0.05).to(DEV)
    gen = torch.Generator(device=DEV).manual_seed(71)
    n = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    taps = {k: (n(H * D, 4) / 2).requires_grad_() for k in "qkv"}
    raw = {k: w[k].detach().reshape(B, T, H * D).clone().requires_grad_() for k in "qkv"}
    gate = n(B, T, H, D).bfloat16()
    nw = torch.ones(D, device=DEV)
    way = n(B, T, H, D).bfloat16()

    mixed = {k: kda.short_conv(raw[k], taps[k])[0].view(B, T, H, D) for k in "qkv"}
    lb = -5.0
    o, _ = kda.chunk_kda(mixed["q"], mixed["k"], mixed["v"], w["g"], w["beta"], w["A_log"],
                         w["dt_bias"].reshape(-1), lower_bound=lb)
    y = kda.gated_norm(o, gate, nw)
    y.backward(way)

    parts = {k: kda.short_conv_fwd(raw[k].detach(), taps[k].detach())[0].view(B, T, H, D) for k in "qkv"}
    dn = kda.gated_norm_bwd(o.detach(), gate, nw, way)
    r = kda.kda_bwd(parts["q"], parts["k"], parts["v"], w["g"], w["beta"], w["A_log"], w["dt_bias"], dn["dx"], lb,
                    D ** -0.5)
    for k in "qkv":
        c = kda.short_conv_bwd(raw[k].detach(), taps[k].detach(), r["d" + k].reshape(B, T, H * D))
        assert torch.equal(raw[k].grad, c["dx"]) and torch.equal(taps[k].grad, c["dweight"]), k


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_convolution_of_single_tokens_has_the_prompts_bits(dtype):
    B, T, C = 3, 40, 72
    w = make(B, T, C, dtype, seed=73)
    x, taps, cb = (w[k].to(DEV) for k in ("x", "taps", "cb"))
    y, state = kda.short_conv_fwd(x, taps, cb)
    _, s = kda.short_conv_fwd(x[:, :25].contiguous(), taps, cb)
    for t in range(25, T):
        c, s = kda.short_conv_decode(x[:, t].contiguous(), taps, s, cb)
        assert torch.equal(c, y[:, t])
    assert torch.equal(s, state)


@pytest.mark.parametrize("final", [True, False])
def test_recurrence_without_gradients_keeps_no_states(final):
    w = make(2, 300, 64, "bf16", seed=79)
    d = {k: t.to(DEV).requires_grad_(k in LEAVES) for k, t in w.items()}
    names = ("x", "g", "gate", "A_log", "dt_bias")
    o, f = kda.gated_scan(*(d[k] for k in names), output_final_state=final)
    assert o.requires_grad
    with torch.no_grad():
        got = kda.gated_scan(*(d[k] for k in names), output_final_state=final)
    plain = kda.gated_scan(*(d[k].detach() for k in names), output_final_state=final)
    for q in (got, plain):
        assert torch.equal(q[0], o) and not q[0].requires_grad
        assert torch.equal(q[1], f) if final else q[1] is None


def test_refusals_on_a_gpu():
    x = torch.zeros(2, 300, 64, dtype=torch.bfloat16, device=DEV)
    p = torch.zeros(64, device=DEV)
    taps = torch.zeros(64, 4, device=DEV)
    side = torch.zeros(2, 64, 300, dtype=torch.bfloat16, device=DEV).transpose(1, 2)
    for call in (lambda: kda.gated_scan_fwd(side, x, x, p, p), lambda: kda.gated_scan_fwd(x, x, side, p, p),
                 lambda: kda.short_conv_fwd(side, taps), lambda: kda.layer_norm_fwd(side, p),
                 lambda: kda.layer_norm_fwd(x, p, residual=side),
                 lambda: kda.short_conv_bwd(x, taps, side), lambda: kda.layer_norm_bwd(x, p, side),
                 lambda: kda.gated_scan_fwd(x, x, x, p[:32], p), lambda: kda.gated_scan_fwd(x, x[:, 1:], x, p, p),
                 lambda: kda.gated_scan_fwd(x, x, x, p, p, initial_state=torch.zeros(3, 64, device=DEV)),
                 lambda: kda.short_conv_fwd(x, taps[:32]), lambda: kda.short_conv_fwd(x, taps, activation="gelu"),
                 lambda: kda.layer_norm_fwd(x, p, residual=x, out=x, sum_out=x),
                 lambda: kda.layer_norm_fwd(x, p, residual=x, out=x, sum_out=x.view(2, 300, 64)),
                 lambda: kda.gated_scan_fwd(x, x, x, p, p, cu_seqlens=torch.zeros(2, dtype=torch.int32, device=DEV)),
                 lambda: kda.gated_scan_decode(x[0], x[0], x[0], p, p, state=torch.zeros(2, 64, device=DEV)),
                 lambda: kda.gated_scan_fwd(x, x, x, p.cpu(), p)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: kda.gated_scan_fwd(x, x.float(), x, p, p), lambda: kda.gated_scan_fwd(x, x, x, p.bfloat16(), p),
                 lambda: kda.short_conv_fwd(x, taps.bfloat16()), lambda: kda.layer_norm_fwd(x, p.half()),
                 lambda: kda.short_conv_decode(x[0], taps, torch.zeros(300, 3, 64, device=DEV)),
                 lambda: kda.gated_scan_fwd(x, x, None, p, p)):
        with pytest.raises(TypeError):
            call()
    few = torch.empty(512, dtype=torch.uint8, device=DEV)
    states = torch.zeros(2 * 38 * 64, device=DEV)
    for call in (lambda: kda.gated_scan_fwd(x, x, x, p, p, workspace=few),
                 lambda: kda.gated_scan_bwd(x, x, x, p, p, x, states, workspace=few),
                 lambda: kda.short_conv_bwd(x, taps, x, workspace=few),
                 lambda: kda.layer_norm_bwd(x, p, x, workspace=few)):
        with pytest.raises(kda.LibKdaError):
            call()
    with pytest.raises(ValueError):
        kda.gated_scan_bwd(x, x, x, p, p, x, states[64:])
    for call in (lambda: kda.short_conv_fwd(x, torch.zeros(64, 5, device=DEV)),
                 lambda: kda.short_conv_fwd(torch.zeros(1, 4, 12, device=DEV), torch.zeros(12, 4, device=DEV)),
                 lambda: kda.layer_norm_fwd(torch.zeros(4, 16392, device=DEV), torch.zeros(16392, device=DEV))):
        with pytest.raises(kda.LibKdaError):
            call()
