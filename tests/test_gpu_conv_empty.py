"""The short convolution of packed batches with very many empty sequences: one behind the
other at the same offset, as where cu_seqlens is padded to a fixed number of sequences."""
import random

import pytest
import torch

import chunked_gated_delta_kda_amd as kda
from block_util import DEV, TYPES
from parity_util import say

pytestmark = pytest.mark.gpu


def make(lens, tail, C, W, dtype, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    lens = torch.tensor(lens)
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
    cu[1:] = lens.cumsum(0)
    T, N, tt = int(cu[-1]) + tail, len(lens), TYPES[dtype]
    return dict(x=n(1, T, C).to(tt), dy=n(1, T, C).to(tt), weight=n(C, W), bias=n(C), h0=n(N, W - 1, C).to(tt),
                dfinal=n(N, W - 1, C).to(tt), cu=cu.to(DEV)), lens


def run(d, cu, h0, dfinal):
    y, f = kda.short_conv_fwd(d["x"], d["weight"], d["bias"], initial_state=h0, cu_seqlens=cu)
    r = kda.short_conv_bwd(d["x"], d["weight"], d["dy"], d["bias"], "silu", h0, dfinal, cu)
    return y, f, r


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("C,W", [(8, 4), (24, 2), (136, 4), (264, 3)])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_the_others_as_without_them(seed, C, W, dtype):
    """Runs of empty sequences in front of, between and behind others of 1 to 40 tokens."""
    rng = random.Random(seed)
    lens = [0] * rng.choice([0, 1, 500])
    for _ in range(rng.randint(1, 30)):
        lens += [rng.randint(1, 40)] + [0] * rng.choice([0, 0, 1, 2, 3, 63, 64, 65, 300, 4096])
    d, lens = make(lens, rng.choice([0, 1, 50]), C, W, dtype, seed)
    y, f, r = run(d, d["cu"], d["h0"], d["dfinal"])
    some = (lens > 0).to(DEV)
    cu = torch.cat([d["cu"][:1], d["cu"][1:][some]])
    say(f"[conv] {len(lens)} sequences, {int(some.sum())} with tokens, C {C} W {W} {dtype}")
    y1, f1, r1 = run(d, cu, d["h0"][some], d["dfinal"][some])
    assert torch.equal(y, y1) and torch.equal(f[some], f1) and torch.equal(f[~some], d["h0"][~some])
    assert torch.equal(r["dh0"][some], r1["dh0"]) and torch.equal(r["dh0"][~some], d["dfinal"][~some])
    for k in ("dx", "dweight", "dbias"):
        assert torch.equal(r[k], r1[k]), k


@pytest.mark.parametrize("tail", [0, 40])
def test_offsets_repeated_a_million_times_cost_little(tail):
    """Passed in a few steps: one by one they are 2^20 loads that wait for each other, some
    200 ms and more.  (Each of them has its state copied: 2^20 workgroups.)"""
    d, lens = make([100] + [0] * (1 << 20) + [60] + [0] * (1 << 20), tail, 72, 4, "bf16", 5)
    run(d, d["cu"], d["h0"], d["dfinal"])
    t = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    torch.cuda.synchronize()
    t[0].record()
    run(d, d["cu"], d["h0"], d["dfinal"])
    t[1].record()
    torch.cuda.synchronize()
    ms = t[0].elapsed_time(t[1])
    say(f"[conv] {len(lens)} sequences: {ms:.2f} ms forward and backward")
    assert ms < 60.0
