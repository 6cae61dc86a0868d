"""Sizes at which the operators around a block have more work items than one dimension of
a grid holds (2^32), or offsets beyond 32 bits."""
import pytest
import torch

import chunked_gated_delta_kda_amd as kda
from parity_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def give_memory_back():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def normal(seed, *shape, dtype=torch.bfloat16):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.empty(*shape, dtype=dtype, device=DEV).normal_(generator=gen)


def test_recurrence_of_2_to_the_23_tiles():
    """Rows of one tile (forward, 2^32 work items of sixteen waves) and of three (gradients),
    of 8 channels; one tensor serves as x, both gates and do."""
    B, T, C = (1 << 22) + 1, 130, 8
    x = normal(1, B, T, C)
    A, bias, h0 = (normal(s, *n, dtype=torch.float32) for s, n in ((2, (C,)), (3, (C,)), (4, (B, C))))
    say(f"[scan] {B} rows of {T} tokens")
    o, f, s = kda.gated_scan_fwd_save(x, x, x, A, bias, h0)
    r = kda.gated_scan_bwd(x, x, x, A, bias, x, s, h0)
    for b in (0, 1 << 21, B - 3):
        p, h = x[b:b + 3].contiguous(), h0[b:b + 3].contiguous()
        o1, f1, s1 = kda.gated_scan_fwd_save(p, p, p, A, bias, h)
        r1 = kda.gated_scan_bwd(p, p, p, A, bias, p, s1, h)
        assert torch.equal(o[b:b + 3], o1) and torch.equal(f[b:b + 3], f1)
        for k in ("dx", "dg", "dinput_gate", "dh0"):
            assert torch.equal(r[k][b:b + 3], r1[k]), k


def test_recurrence_of_2_to_the_23_tiles_that_wait():
    B, T, C = (1 << 21) + 1, 500, 8
    x = normal(5, B, T, C)
    A, bias = normal(6, C, dtype=torch.float32), normal(7, C, dtype=torch.float32)
    say(f"[scan] {B} rows of {T} tokens")
    o, f = kda.gated_scan_fwd(x, x, x, A, bias)
    for b in (0, 1 << 20, B - 3):
        p = x[b:b + 3].contiguous()
        o1, f1 = kda.gated_scan_fwd(p, p, p, A, bias)
        assert torch.equal(o[b:b + 3], o1) and torch.equal(f[b:b + 3], f1)


def test_states_of_2_to_the_24_empty_sequences():
    """A workgroup each, and a few tokens in between."""
    N, C, T = (1 << 24) + 7, 8, 300
    cu = torch.zeros(N + 1, dtype=torch.int32, device=DEV)
    cu[N // 2:] = 200
    cu[N:] = 300
    x = normal(8, 1, T, C)
    A, bias, h0 = (normal(s, *n, dtype=torch.float32) for s, n in ((9, (C,)), (10, (C,)), (11, (N, C))))
    few = torch.tensor([0, 200, 300], dtype=torch.int32, device=DEV)
    at = torch.tensor([N // 2 - 1, N - 1], device=DEV)
    rest = torch.ones(N, dtype=torch.bool, device=DEV)
    rest[at] = False
    say(f"[scan] {N} sequences")
    o, f = kda.gated_scan_fwd(x, x, x, A, bias, h0, cu_seqlens=cu)
    ow, fw = kda.gated_scan_fwd(x, x, x, A, bias, h0[at].contiguous(), cu_seqlens=few)
    assert torch.equal(o, ow) and torch.equal(f[at], fw) and torch.equal(f[rest], h0[rest])
    say(f"[conv] {N} sequences")
    taps = normal(12, C, 2, dtype=torch.float32)
    s0 = h0.bfloat16().view(N, 1, C)
    y, f = kda.short_conv_fwd(x, taps, initial_state=s0, cu_seqlens=cu)
    yw, fw = kda.short_conv_fwd(x, taps, initial_state=s0[at].contiguous(), cu_seqlens=few)
    assert torch.equal(y, yw) and torch.equal(f[at], fw) and torch.equal(f[rest], s0[rest])


def test_single_tokens_of_2_to_the_24_workgroups():
    """2^32 channels in all, fp32; one tensor serves as x and both gates."""
    N, C = (1 << 20) + 1, 4096
    x, state = normal(13, N, C, dtype=torch.float32), normal(14, N, C, dtype=torch.float32)
    A, bias = normal(15, C, dtype=torch.float32), normal(16, C, dtype=torch.float32)
    at = [0, (1 << 19) - 1, N - 2]
    say(f"[scan] single tokens of {N} sequences")
    before = [state[i:i + 2].clone() for i in at]
    o, s = kda.gated_scan_decode(x, x, x, A, bias, state, state_out=state)
    for i, b in zip(at, before):
        p = x[i:i + 2].contiguous()
        ow, sw = kda.gated_scan_decode(p, p, p, A, bias, b)
        assert torch.equal(o[i:i + 2], ow) and torch.equal(s[i:i + 2], sw)
    del o
    say(f"[conv] single tokens of {N} sequences")
    taps = normal(17, C, 2, dtype=torch.float32)
    y, s = kda.short_conv_decode(x, taps, state.view(N, 1, C))
    for i in at:
        yw, sw = kda.short_conv_decode(x[i:i + 2].contiguous(), taps, state[i:i + 2].view(2, 1, C).clone())
        assert torch.equal(y[i:i + 2], yw) and torch.equal(s[i:i + 2], sw)
    assert torch.equal(s.view(N, C), x)


def test_convolution_of_2_to_the_24_workgroups():
    """dweight of an identity with dy = x: sums of products of tokens, each product and
    partial sum of fp32 off by 2^-24 of itself, 64 tokens of one sign to a partial sum."""
    T, C = (1 << 30) + 100, 8
    x = normal(18, 1, T, C, dtype=torch.float32)
    taps = normal(19, C, 2, dtype=torch.float32)
    say(f"[conv] {T} tokens")
    y, f = kda.short_conv_fwd(x, taps, activation="none")
    for t in (1, (1 << 29) - 3, T - 50):
        p = x[:, t - 1:t + 50].contiguous()
        assert torch.equal(y[:, t:t + 50], kda.short_conv_fwd(p, taps, activation="none")[0][:, 1:])
    assert torch.equal(f[0, 0], x[0, -1])
    del y
    say(f"[conv] gradients of {T} tokens")
    r = kda.short_conv_bwd(x, taps, x, activation="none")
    for t in (1, (1 << 29) - 3, T - 50):
        p = x[:, t:t + 50].contiguous()
        assert torch.equal(r["dx"][:, t:t + 49], kda.short_conv_bwd(p, taps, p, activation="none")["dx"][:, :49])
    want = torch.zeros(2, C, dtype=torch.float64, device=DEV)
    size = torch.zeros(2, C, dtype=torch.float64, device=DEV)
    for t in range(0, T, 1 << 24):
        q = x[0, t:t + (1 << 24)].double()
        before = x[0, t - 1:t - 1 + len(q)].double() if t else torch.cat([torch.zeros_like(q[:1]), q[:-1]])
        for j, v in enumerate((q * before, q * q)):
            want[j] += v.sum(0)
            size[j] += v.abs().sum(0)
    assert ((r["dweight"].double().t() - want).abs() <= 65 * 2.0 ** -24 * size + want.abs() * 2.0 ** -24).all()


def test_layer_norm_of_2_to_the_32_elements():
    rows, D = (1 << 20) + 3, 4104
    x = normal(20, rows, D)
    w = normal(21, D, dtype=torch.float32)
    say(f"[norm] {rows} rows of {D}")
    y, _ = kda.layer_norm_fwd(x, w, w)
    r = kda.layer_norm_bwd(x, w, x)
    for i in (0, (1 << 19) - 5, rows - 10):
        p = x[i:i + 10].contiguous()
        assert torch.equal(y[i:i + 10], kda.layer_norm_fwd(p, w, w)[0])
        assert torch.equal(r["dx"][i:i + 10], kda.layer_norm_bwd(p, w, p)["dx"])


def test_rows_of_2_to_the_20_channels():
    """The widest rows, 2^31 bytes and more of them: as their blocks of channels alone."""
    T, C = 1100, 1 << 20
    x = normal(22, 1, T, C)
    A, bias = normal(23, C, dtype=torch.float32), normal(24, C, dtype=torch.float32)
    taps = normal(25, C, 4, dtype=torch.float32)
    say(f"[scan] {T} tokens of {C}")
    o, f, s = kda.gated_scan_fwd_save(x, x, x, A, bias)
    r = kda.gated_scan_bwd(x, x, x, A, bias, x, s)
    say(f"[conv] {T} tokens of {C}")
    y, _ = kda.short_conv_fwd(x, taps)
    g = kda.short_conv_bwd(x, taps, x)
    for c in (0, C // 2 + 128, C - 128):
        cut = slice(c, c + 128)
        p, a, b, w = x[..., cut].contiguous(), A[cut].contiguous(), bias[cut].contiguous(), taps[cut].contiguous()
        o1, f1, s1 = kda.gated_scan_fwd_save(p, p, p, a, b)
        assert torch.equal(o[..., cut], o1) and torch.equal(f[:, cut], f1)
        r1 = kda.gated_scan_bwd(p, p, p, a, b, p, s1)
        for k in ("dx", "dg", "dinput_gate", "dA_log", "ddt_bias", "dh0"):
            assert torch.equal(r[k][..., cut], r1[k]), k
        assert torch.equal(y[..., cut], kda.short_conv_fwd(p, w)[0])
        assert torch.equal(g["dx"][..., cut], kda.short_conv_bwd(p, w, p)["dx"])


def test_sizes_beyond_32_bits_are_refused():
    x = torch.empty(1, (1 << 32) + 5, 8, dtype=torch.bfloat16, device=DEV)  # (5 tokens in 32 bits)
    p = torch.zeros(8, device=DEV)
    for call in (lambda: kda.gated_scan_fwd(x, x, x, p, p), lambda: kda.short_conv_fwd(x, torch.zeros(8, 4, device=DEV)),
                 lambda: kda.gated_scan_decode(x[0], x[0], x[0], p, p), lambda: kda.layer_norm_fwd(x, p)):
        with pytest.raises(kda.LibKdaError):
            call()


def test_the_longest_row():
    """2^31 - 65 tokens: its end is that of the last tokens alone, behind the state (or the
    tokens) in front of them."""
    T, C, n = (1 << 31) - 65, 8, 300
    x = normal(26, 1, T, C)
    A, bias = normal(27, C, dtype=torch.float32), normal(28, C, dtype=torch.float32)
    taps = normal(29, C, 4, dtype=torch.float32)
    say(f"[conv] {T} tokens")
    y, f = kda.short_conv_fwd(x, taps)
    end = x[:, T - n:].contiguous()
    yw, fw = kda.short_conv_fwd(end, taps, initial_state=x[:, T - n - 3:T - n].contiguous())
    assert torch.equal(y[:, T - n:], yw) and torch.equal(f, fw)
    del y
    say(f"[scan] {T} tokens")
    o, f = kda.gated_scan_fwd(x, x, x, A, bias)
    ow, fw = kda.gated_scan_fwd(end, end, end, A, bias, initial_state=o[:, T - n - 1].float().contiguous())
    # the state in front comes rounded to bf16, and decays; outputs are rounded, too
    assert ((o[:, T - n:].float() - ow.float()).abs() <= 2.0 ** -7 * (ow.float().abs() + fw.abs().max() + 1)).all()
    assert torch.isfinite(f).all() and (f - fw).abs().max() <= 2.0 ** -7 * (fw.abs().max() + 1)
