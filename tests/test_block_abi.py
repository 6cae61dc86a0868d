"""gated_scan_*, short_conv_* and layer_norm_* on the host: every refusal comes
before any HIP call (fake pointers, no device), and so do the wrappers'."""
import ctypes

import pytest
import torch

import chunked_gated_delta_kda_amd as kda

FAKE = ctypes.c_void_p(0x1000)
BIG = 1 << 62
odd = lambda n: ctypes.c_void_p(0x1000 + n)  # noqa: E731


@pytest.fixture(scope="module")
def lib():
    return kda.load()


def call(fn, base, over):
    assert set(over) <= set(base)
    return fn(*{**base, **over}.values())


SIZES = [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(C=0), 1), (dict(C=12), 2), (dict(C=(1 << 20) + 8), 2), (dict(dtype=2), 1),
    (dict(dtype=-1), 1), (dict(B=1 << 16, T=1 << 15), 1), (dict(T=(1 << 31) - 64, C=8), 1), (dict(cu=FAKE, B=2, N=2), 1), (dict(cu=FAKE, N=0), 1),
    (dict(cu=odd(2)), 1), (dict(x=None), 1), (dict(x=odd(8)), 1), (dict(h0=odd(8)), 1)]

SCAN = dict(x=FAKE, g=FAKE, gate=FAKE, A=FAKE, b=FAKE, h0=None, hT=None, cu=None, N=1, dtype=0, B=1, T=300, C=64, o=FAKE,
            states=None, ws=FAKE, wsb=BIG, stream=None)
SCAN_ONLY = [(dict(g=None), 1), (dict(gate=None), 1), (dict(A=None), 1), (dict(b=None), 1), (dict(g=odd(4)), 1),
             (dict(gate=odd(8)), 1), (dict(A=odd(2)), 1), (dict(b=odd(1)), 1), (dict(ws=None), 3),
             (dict(ws=odd(16)), 3), (dict(wsb=255), 3), (dict(states=odd(8)), 1),
             (dict(B=1 << 24, T=64, C=1 << 13), 1)]


@pytest.mark.parametrize("over,code", SIZES + SCAN_ONLY + [(dict(o=None), 1), (dict(o=odd(8)), 1),
                                                           (dict(hT=odd(4)), 1)])
def test_gated_scan_fwd_rejects_on_host(lib, over, code):
    assert call(lib.gated_scan_fwd, SCAN, over) == code


SCAN_BWD = dict(x=FAKE, g=FAKE, gate=FAKE, A=FAKE, b=FAKE, h0=None, cu=None, N=1, dtype=0, B=1, T=300, C=64, do=FAKE,
                df=None, states=FAKE, dx=FAKE, dg=FAKE, di=FAKE, dA=FAKE, db=FAKE, dh0=None, ws=FAKE, wsb=BIG,
                stream=None)


@pytest.mark.parametrize("over,code", SIZES + SCAN_ONLY + [
    ({n: None}, 1) for n in ("do", "states", "dx", "dg", "di", "dA", "db")] + [
    ({n: odd(8)}, 1) for n in ("do", "df", "dx", "dg", "di", "dh0")] + [(dict(dA=odd(2)), 1), (dict(db=odd(2)), 1)])
def test_gated_scan_bwd_rejects_on_host(lib, over, code):
    assert call(lib.gated_scan_bwd, SCAN_BWD, over) == code


SCAN_TOK = dict(x=FAKE, g=FAKE, gate=FAKE, A=FAKE, b=FAKE, s_in=None, s_out=FAKE, dtype=0, N=2, C=64, o=FAKE,
                stream=None)


@pytest.mark.parametrize("over,code", [({n: None}, 1) for n in ("x", "g", "gate", "A", "b", "s_out", "o")] + [
    ({n: odd(8)}, 1) for n in ("x", "g", "gate", "s_in", "s_out", "o")] + [
    (dict(N=0), 1), (dict(C=20), 2), (dict(dtype=7), 1), (dict(A=odd(2)), 1)])
def test_gated_scan_decode_rejects_on_host(lib, over, code):
    assert call(lib.gated_scan_decode, SCAN_TOK, over) == code


CONV = dict(x=FAKE, w=FAKE, b=None, act=1, h0=None, hT=None, cu=None, N=1, dtype=0, B=1, T=16, C=64, W=4, y=FAKE,
            stream=None)
CONV_ONLY = [(dict(w=None), 1), (dict(w=odd(2)), 1), (dict(b=odd(2)), 1), (dict(act=2), 1), (dict(act=-1), 1),
             (dict(W=1), 2), (dict(W=5), 2), (dict(B=1 << 23, T=64, C=1 << 15), 1)]


@pytest.mark.parametrize("over,code", SIZES + CONV_ONLY + [(dict(y=None), 1), (dict(y=odd(8)), 1),
                                                           (dict(hT=odd(8)), 1)])
def test_short_conv_fwd_rejects_on_host(lib, over, code):
    assert call(lib.short_conv_fwd, CONV, over) == code


CONV_BWD = dict(x=FAKE, w=FAKE, b=None, act=1, h0=None, cu=None, N=1, dtype=0, B=1, T=16, C=64, W=4, dy=FAKE, df=None,
                dx=FAKE, dw=FAKE, db=None, dh0=None, ws=FAKE, wsb=BIG, stream=None)


@pytest.mark.parametrize("over,code", SIZES + CONV_ONLY + [
    (dict(dy=None), 1), (dict(dx=None), 1), (dict(dw=None), 1), (dict(b=FAKE), 1), (dict(dy=odd(8)), 1),
    (dict(dx=odd(8)), 1), (dict(df=odd(8)), 1), (dict(dh0=odd(8)), 1), (dict(dw=odd(2)), 1), (dict(ws=None), 3),
    (dict(ws=odd(16)), 3), (dict(wsb=255), 3)])
def test_short_conv_bwd_rejects_on_host(lib, over, code):
    assert call(lib.short_conv_bwd, CONV_BWD, over) == code


CONV_TOK = dict(x=FAKE, w=FAKE, b=None, act=1, s_in=FAKE, s_out=FAKE, dtype=0, N=2, C=64, W=4, y=FAKE, stream=None)


@pytest.mark.parametrize("over,code", CONV_ONLY[:-1] + [({n: None}, 1) for n in ("x", "s_in", "s_out", "y")] + [
    ({n: odd(8)}, 1) for n in ("x", "s_in", "s_out", "y")] + [(dict(N=0), 1), (dict(C=4), 2), (dict(dtype=2), 1)])
def test_short_conv_decode_rejects_on_host(lib, over, code):
    assert call(lib.short_conv_decode, CONV_TOK, over) == code


NORM = dict(x=FAKE, res=None, w=FAKE, b=None, eps=1e-5, dtype=0, rows=4, D=64, y=FAKE, sum=None, stream=None)
NORM_ONLY = [(dict(rows=-1), 1), (dict(rows=1 << 31), 1), (dict(D=0), 1), (dict(D=12), 2), (dict(D=16392), 2),
             (dict(dtype=2), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
             (dict(w=None), 1), (dict(w=odd(2)), 1)]


@pytest.mark.parametrize("over,code", NORM_ONLY + [
    (dict(x=None), 1), (dict(y=None), 1), (dict(res=FAKE), 1), (dict(x=odd(8)), 1), (dict(y=odd(8)), 1),
    (dict(res=odd(8), sum=FAKE), 1), (dict(res=FAKE, sum=odd(8)), 1), (dict(b=odd(2)), 1),
    (dict(res=FAKE, sum=FAKE), 1)])
def test_layer_norm_fwd_rejects_on_host(lib, over, code):
    assert call(lib.layer_norm_fwd, NORM, over) == code


NORM_BWD = dict(sum=FAKE, w=FAKE, eps=1e-5, dtype=0, rows=4, D=64, dy=FAKE, ds=None, dx=FAKE, dw=FAKE, db=None, ws=FAKE,
                wsb=BIG, stream=None)


@pytest.mark.parametrize("over,code", NORM_ONLY + [
    (dict(sum=None), 1), (dict(dy=None), 1), (dict(dx=None), 1), (dict(dw=None), 1), (dict(sum=odd(8)), 1),
    (dict(dy=odd(8)), 1), (dict(ds=odd(8)), 1), (dict(dx=odd(8)), 1), (dict(dw=odd(2)), 1), (dict(db=odd(2)), 1),
    (dict(ws=None), 3), (dict(ws=odd(16)), 3), (dict(wsb=255), 3)])
def test_layer_norm_bwd_rejects_on_host(lib, over, code):
    assert call(lib.layer_norm_bwd, NORM_BWD, over) == code


def test_no_rows_is_no_call(lib):
    assert call(lib.layer_norm_fwd, NORM, dict(rows=0, x=None, y=None)) == 0


def test_sizes(lib):
    assert lib.gated_scan_states(2, 129, 64) == 2 * 17 * 64
    assert lib.gated_scan_states(1, 0, 64) == 0
    assert lib.gated_scan_states(1, (1 << 31) - 65, 8) == ((1 << 31) - 64) // 8 * 8
    for bad in ((0, 1, 64), (1, -1, 64), (1, (1 << 31) - 64, 8), (1, 1, 12), (1, 1, (1 << 20) + 8), (1 << 16, 1 << 15, 64)):
        assert lib.gated_scan_states(*bad) == -1
        assert kda.gated_scan_workspace_size(*bad) == kda.gated_scan_workspace_size(*bad, backward=True) == 0
        assert lib.short_conv_bwd_workspace_size(0, *bad, 4) == 0
    # more tiles than tickets: 2^24 of 64 tokens, 2^7 blocks of 64 channels
    assert lib.gated_scan_states(1 << 24, 64, 1 << 13) == -1
    assert kda.gated_scan_workspace_size(1 << 24, 64, 1 << 13) == 0
    assert lib.gated_scan_states((1 << 24) - 1, 64, 1 << 13) == ((1 << 24) - 1) << 16
    # rows of one tile need none, packed ones their tables, longer ones words for every tile
    assert kda.gated_scan_workspace_size(2, 256, 64) == 256
    assert kda.gated_scan_workspace_size(1, 256, 64, packed=True) > 256
    assert kda.gated_scan_workspace_size(2, 100, 64, packed=True) == 0
    assert kda.gated_scan_workspace_size(2, 257, 64) >= 2 * 3 * 64 * 8
    assert kda.gated_scan_workspace_size(2, 257, 64, True) >= 2 * 5 * 64 * 8 + 2 * 5 * 2 * 64 * 4
    assert lib.short_conv_bwd_workspace_size(0, 1 << 23, 64, 1 << 15, 4) == 0  # workgroups
    assert lib.short_conv_bwd_workspace_size(0, 1, 1, 64, 5) == lib.short_conv_bwd_workspace_size(2, 1, 1, 64, 4) == 0
    assert lib.layer_norm_bwd_workspace_size(0, 5, 12) == lib.layer_norm_bwd_workspace_size(3, 5, 64) == 0
    assert lib.layer_norm_bwd_workspace_size(0, 1 << 31, 64) == lib.layer_norm_bwd_workspace_size(1, 5, 16392) == 0


def test_wrappers_refuse_what_is_not_on_a_gpu_or_of_another_type():
    x = torch.zeros(1, 4, 8, dtype=torch.bfloat16)
    p = torch.zeros(8)
    with pytest.raises(ValueError, match="GPU"):
        kda.gated_scan_fwd(x, x, x, p, p)
    with pytest.raises(ValueError, match="GPU"):
        kda.short_conv_fwd(x, torch.zeros(8, 4))
    with pytest.raises(ValueError, match="GPU"):
        kda.layer_norm_fwd(x, p)
    for bad in (x.half(), x.double()):
        with pytest.raises(TypeError, match="float32"):
            kda.gated_scan_fwd(bad, bad, bad, p, p)
        with pytest.raises(TypeError, match="float32"):
            kda.short_conv_decode(bad[0], torch.zeros(8, 4), bad)
        with pytest.raises(TypeError, match="float32"):
            kda.layer_norm_bwd(bad, p, bad)
    with pytest.raises(TypeError, match="Tensor"):
        kda.layer_norm_fwd(None, p)
