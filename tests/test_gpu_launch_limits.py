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
