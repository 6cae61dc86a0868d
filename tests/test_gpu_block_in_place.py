"""Calls around a block whose output is one of their inputs, and those that are refused
since their workgroups read what others write."""
import pytest
import torch

import chunked_gated_delta_kda_amd as kda
from block_util import DEV, offsets, to_gpu
from test_gpu_conv import make as make_conv
from test_gpu_scan import args
from test_gpu_scan import make as make_scan

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", ["x", "g", "gate"])
@pytest.mark.parametrize("B,T,lens", [(2, 100, None), (3, 256, None), (2, 1500, None), (1, 0, [70, 0, 1, 500, 3])])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_the_recurrence_over_one_of_its_inputs(dtype, B, T, lens, which):
    cu = None if lens is None else offsets(lens)
    d = to_gpu(make_scan(B, T or int(cu[-1]) + 7, 72, seed=201, dtype=dtype, cu=cu))
    o, f, s = kda.gated_scan_fwd_save(*args(d), d["h0"], cu_seqlens=d["cu"])
    o2, f2, s2 = kda.gated_scan_fwd_save(*args(d), d["h0"], cu_seqlens=d["cu"], out=d[which])
    assert o2 is d[which] and torch.equal(o, o2) and torch.equal(f, f2) and torch.equal(s, s2)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_single_tokens_over_their_input(dtype):
    d = to_gpu(make_scan(5, 1, 360, seed=203, dtype=dtype))
    tok = [d[k][:, 0].contiguous() for k in ("x", "g", "gate")]
    o, s = kda.gated_scan_decode(*tok, d["A_log"], d["dt_bias"], d["h0"])
    for k in range(3):
        q = [t.clone() for t in tok]
        state = d["h0"].clone()
        o2, s2 = kda.gated_scan_decode(*q, d["A_log"], d["dt_bias"], state, state_out=state, out=q[k])
        assert o2 is q[k] and s2 is state and torch.equal(o, o2) and torch.equal(s, s2)
    for N, C in ((5, 360), (64, 4096)):
        w = to_gpu(make_conv(N, 1, C, seed=207, dtype=dtype))
        x, state = w["x"][:, 0].contiguous(), w["h0"].clone()
        y, s = kda.short_conv_decode(x, w["weight"], state, w["bias"])
        y2, s2 = kda.short_conv_decode(x, w["weight"], state, w["bias"], state_out=state, out=x)
        assert y2 is x and s2 is state and torch.equal(y, y2) and torch.equal(s, s2)


def test_refusals():
    room = torch.zeros(1, 301, 64, device=DEV)
    x, behind = room[:, :300], room[:, 1:]
    other = torch.zeros(1, 300, 64, device=DEV)
    p, taps, h0, cs = (torch.zeros(*s, device=DEV) for s in ((64,), (64, 4), (1, 64), (1, 3, 64)))
    for call in (lambda: kda.short_conv_fwd(x, taps, out=x), lambda: kda.short_conv_fwd(x, taps, out=behind),
                 lambda: kda.short_conv_fwd(other, taps, initial_state=cs, final_out=cs),
                 lambda: kda.gated_scan_fwd(x, other, other, p, p, out=behind),
                 lambda: kda.gated_scan_fwd(other, other, x, p, p, out=behind),
                 lambda: kda.gated_scan_fwd(other, other, other, p, p, initial_state=h0, final_out=h0),
                 lambda: kda.gated_scan_decode(x[0], other[0], other[0], p, p, out=behind[0]),
                 lambda: kda.gated_scan_decode(other[0], other[0], other[0], p, p, state=x[0], state_out=behind[0]),
                 lambda: kda.gated_scan_decode(x[0], other[0], other[0], p, p, state_out=x[0]),
                 lambda: kda.short_conv_decode(x[0], taps, torch.zeros(300, 3, 64, device=DEV), out=behind[0]),
                 lambda: kda.layer_norm_fwd(x, p, out=behind), lambda: kda.layer_norm_fwd(x, p, residual=behind, out=x),
                 lambda: kda.layer_norm_fwd(other, p, residual=other, out=x, sum_out=behind)):
        with pytest.raises(kda.LibKdaError):
            call()
    # beside each other, and over an input, they are not
    kda.short_conv_fwd(x, taps, out=other)
    kda.gated_scan_fwd(x, other, other, p, p, out=other)
    torch.cuda.synchronize()
