"""Sizes at which a launch has more work items than one dimension of a grid holds
(2^32): linear attention and the gated norm take them, as their limits say."""
import pytest
import torch

import chunked_gated_delta_kda_amd as kda
from parity_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = 2.0 ** -8 * 1.02  # a rounding to bf16, inside or at the end (see test_gpu_linear)


@pytest.fixture(autouse=True)
def give_memory_back():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def normal(gen, *shape):
    return torch.empty(*shape, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)


def test_linear_attention_of_2_to_the_23_pairs():
    """One token each, no states: o = scale (q k) v, dv = scale (q k) do,
    dk = scale (do v) q, dq = scale (do v) k, each with a rounding of the product in
    brackets (or of its factor) and one of the result."""
    B, H, D = (1 << 17) + 3, 64, 64  # 2^23 + 192 workgroups of 512 threads
    gen = torch.Generator(device=DEV).manual_seed(1)
    q, k, v, do = (normal(gen, B, 1, H, D) for _ in range(4))
    ld = torch.full((H,), -0.3, device=DEV)
    say(f"[la] {B} sequences of one token, {H} heads")
    o, S = kda.la_fwd(q, k, v, ld, output_final_state=False)
    r = kda.la_bwd(q, k, v, ld, do, need_dh0=False)
    assert S is None and r["dh0"] is None
    scale = D ** -0.5

    def near(name, got, a, b, c):
        for i in range(0, B, 1 << 14):
            a_, b_, c_ = (t[i:i + (1 << 14)].float() for t in (a, b, c))
            want = scale * (a_ * b_).sum(-1, keepdim=True) * c_
            mag = scale * (a_ * b_).abs().sum(-1, keepdim=True) * c_.abs()
            over = (got[i:i + (1 << 14)].float() - want).abs() - BF * (mag + want.abs()) - 1e-30
            assert over.max() <= 0, (name, i)  # (a NaN fails too)

    near("o", o, q, k, v)
    near("dv", r["dv"], q, k, do)
    near("dk", r["dk"], do, v, q)
    near("dq", r["dq"], do, v, k)


def test_segments_of_2_to_the_22_states():
    """The scan over segments has a work item for every four elements of a state: here
    2^32, nearly all of empty sequences."""
    H, D, N = 64, 64, 1 << 16
    lens = {5: 200, N - 1: 170}
    T = sum(lens.values())
    cu = torch.zeros(N + 1, dtype=torch.int32)
    cu[6:] = 200
    cu[N] = T
    gen = torch.Generator(device=DEV).manual_seed(2)
    q, k, v = (normal(gen, 1, T, H, D) for _ in range(3))
    ld = torch.full((H,), -0.02, device=DEV)
    ws = torch.empty(kda.la_workspace_size(1, T, H, D, D, N, 1), dtype=torch.uint8, device=DEV)
    say(f"[la] {N} sequences, {H} heads, {ws.numel() / 2 ** 30:.0f} GiB of segments' states")
    ws.fill_(255)
    o, _ = kda.la_fwd(q, k, v, ld, cu_seqlens=cu.to(DEV), output_final_state=False, workspace=ws,
                      segment_chunks=1)
    few = torch.tensor([0, 200, T], dtype=torch.int32, device=DEV)
    want, _ = kda.la_fwd(q, k, v, ld, cu_seqlens=few, output_final_state=False, segment_chunks=1)
    assert torch.equal(o, want)


def test_gated_norm_of_2_to_the_26_rows():
    """64 lanes a row: 2^32 work items, in place."""
    rows, D = (1 << 26) + 70, 264
    gen = torch.Generator(device=DEV).manual_seed(3)
    x = normal(gen, rows, 1, D)
    w = torch.randn(D, generator=gen, device=DEV)
    at = [0, (1 << 25) - 3, (1 << 26) - 50, rows - 100]
    say(f"[norm] {rows} rows of {D}")
    want = [kda.gated_norm_fwd(x[i:i + 100].clone(), None, w) for i in at]
    kda.gated_norm_fwd(x, None, w, out=x)
    for i, y in zip(at, want):
        assert torch.equal(x[i:i + 100], y), i


def test_gated_norm_gradients_of_2_to_the_24_heads():
    """A workgroup for each head's sum."""
    H, D = (1 << 24) + 6, 8
    gen = torch.Generator(device=DEV).manual_seed(4)
    x, gate, res, dy = (normal(gen, 1, H, D) for _ in range(4))
    w, rs = torch.randn(D, generator=gen, device=DEV), torch.randn(H, generator=gen, device=DEV)
    say(f"[norm] one token, {H} heads of {D}")
    r = kda.gated_norm_bwd(x, gate, w, dy, "silu", residual=res, residual_scale=rs)
    for s in (slice(0, H // 2), slice(H // 2, H)):
        half = [t[:, s].contiguous() for t in (x, gate, dy, res)]
        h = kda.gated_norm_bwd(half[0], half[1], w, half[2], "silu", residual=half[3],
                               residual_scale=rs[s].contiguous())
        for n in ("dx", "dgate", "dresidual"):
            assert torch.equal(r[n][:, s], h[n]), n
        assert torch.equal(r["dresidual_scale"][s], h["dresidual_scale"])


def test_decode_of_2_to_the_24_pairs():
    """256 GiB of states, updated in place."""
    N, H, D = (1 << 18) + 1, 64, 64
    free = torch.cuda.mem_get_info()[0]
    if free < (N * H * D * (D * 4 + 8) + (2 << 30)):
        pytest.skip(f"{free / 2 ** 30:.0f} GiB of device memory are free")
    gen = torch.Generator(device=DEV).manual_seed(5)
    q, k, v = (normal(gen, N, H, D) for _ in range(3))
    ld = torch.full((H,), -0.3, device=DEV)
    state = torch.full((N, H, D, D), 0.5, device=DEV)
    say(f"[la] {N} sequences, {H} heads, {state.numel() * 4 / 2 ** 30:.0f} GiB of states")
    o, S = kda.la_decode(q, k, v, ld, state=state, state_out=state)
    for i in (0, 1 << 17, N - 2, N - 1):
        one = [t[i:i + 1].contiguous() for t in (q, k, v)]
        ow, Sw = kda.la_decode(*one, ld, state=torch.full((1, H, D, D), 0.5, device=DEV))
        assert torch.equal(o[i:i + 1], ow) and torch.equal(S[i:i + 1], Sw), i
