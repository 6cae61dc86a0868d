"""Outputs that share memory with inputs, with each other or with the workspace: refused on
the host before any HIP call (addresses that are never read, no device).  What may be in
place is run in test_gpu_block_in_place.py."""
import ctypes

import pytest

import chunked_gated_delta_kda_amd as kda

BIG = 1 << 30  # bytes between two arrays, and the workspace's


@pytest.fixture(scope="module")
def lib():
    return kda.load()


def arrays(names):
    return {n: (i + 1) << 32 for i, n in enumerate(names.split())}


def refused(fn, order, base, over):
    at = {**base, **over}
    return fn(*(ctypes.c_void_p(at[n]) if isinstance(at[n], int) and at[n] > 1 << 30 else at[n] for n in order)) == 1


def cases(outs, ins, may):
    """(output, what it shares memory with, bytes behind that one's beginning)"""
    r = []
    for o in outs:
        for i in [n for n in outs if n != o] + ins:
            if (o, i) not in may:
                r.append((o, i, 0))
            r += [(o, i, 16), (o, i, -16)]  # (one's beginning inside the other)
    return r


def shift(base, case):
    o, i, d = case
    return {o: base[i] + d}


T, C, W, N = 100, 64, 4, 3
SCAN = arrays("x g gate A b h0 hT cu o states ws")
SCAN_ORDER = "x g gate A b h0 hT cu n dt B T C o states ws wsb stream".split()
SCAN_REST = dict(n=N, dt=0, B=1, T=T, C=C, wsb=BIG, stream=None)


@pytest.mark.parametrize("case", [c for c in cases(["o", "hT", "states"], ["x", "g", "gate", "h0"],
                                                   [("o", "x"), ("o", "g"), ("o", "gate")])], ids=str)
def test_gated_scan_fwd(lib, case):
    assert refused(lib.gated_scan_fwd, SCAN_ORDER, {**SCAN, **SCAN_REST}, shift(SCAN, case))


@pytest.mark.parametrize("o", ["o", "hT", "states"])
@pytest.mark.parametrize("i", ["A", "b", "cu"])
def test_gated_scan_fwd_parameters(lib, o, i):
    assert refused(lib.gated_scan_fwd, SCAN_ORDER, {**SCAN, **SCAN_REST}, {o: SCAN[i]})


@pytest.mark.parametrize("i", ["x", "g", "gate", "A", "b", "h0", "hT", "cu", "o", "states"])
def test_gated_scan_fwd_workspace(lib, i):
    assert refused(lib.gated_scan_fwd, SCAN_ORDER, {**SCAN, **SCAN_REST}, dict(ws=SCAN[i]))


BWD = arrays("x g gate A b h0 cu do df states dx dg di dA db dh0 ws")
BWD_ORDER = "x g gate A b h0 cu n dt B T C do df states dx dg di dA db dh0 ws wsb stream".split()


@pytest.mark.parametrize("case", cases(["dx", "dg", "di", "dA", "db", "dh0"], ["x", "g", "gate", "do", "h0", "df", "states"],
                                       [(o, i) for o in ("dx", "dg", "di") for i in ("x", "g", "gate", "do")]), ids=str)
def test_gated_scan_bwd(lib, case):
    assert refused(lib.gated_scan_bwd, BWD_ORDER, {**BWD, **SCAN_REST}, shift(BWD, case))


@pytest.mark.parametrize("i", [n for n in BWD if n != "ws"])
def test_gated_scan_bwd_workspace(lib, i):
    assert refused(lib.gated_scan_bwd, BWD_ORDER, {**BWD, **SCAN_REST}, dict(ws=BWD[i]))


TOK = arrays("x g gate A b s_in s_out o")
TOK_ORDER = "x g gate A b s_in s_out dt N C o stream".split()


@pytest.mark.parametrize("case", cases(["o", "s_out"], ["x", "g", "gate", "s_in"],
                                       [("o", "x"), ("o", "g"), ("o", "gate"), ("s_out", "s_in")]), ids=str)
def test_gated_scan_decode(lib, case):
    assert refused(lib.gated_scan_decode, TOK_ORDER, dict(TOK, dt=0, N=N, C=C, stream=None), shift(TOK, case))


CONV = arrays("x w b h0 hT cu y")
CONV_ORDER = "x w b act h0 hT cu n dt B T C W y stream".split()
CONV_REST = dict(act=1, n=N, dt=0, B=1, T=T, C=C, W=W, wsb=BIG, stream=None)


@pytest.mark.parametrize("case", cases(["y", "hT"], ["x", "h0", "w", "b"], []), ids=str)
def test_short_conv_fwd(lib, case):
    assert refused(lib.short_conv_fwd, CONV_ORDER, {**CONV, **CONV_REST}, shift(CONV, case))


CBWD = arrays("x w b h0 cu dy df dx dw db dh0 ws")
CBWD_ORDER = "x w b act h0 cu n dt B T C W dy df dx dw db dh0 ws wsb stream".split()


@pytest.mark.parametrize("case", cases(["dx", "dh0", "dw", "db"], ["x", "h0", "dy", "df", "w", "b"], []), ids=str)
def test_short_conv_bwd(lib, case):
    assert refused(lib.short_conv_bwd, CBWD_ORDER, {**CBWD, **CONV_REST}, shift(CBWD, case))


@pytest.mark.parametrize("i", [n for n in CBWD if n != "ws"])
def test_short_conv_bwd_workspace(lib, i):
    assert refused(lib.short_conv_bwd, CBWD_ORDER, {**CBWD, **CONV_REST}, dict(ws=CBWD[i]))


CTOK = arrays("x w b s_in s_out y")
CTOK_ORDER = "x w b act s_in s_out dt N C W y stream".split()


@pytest.mark.parametrize("case", cases(["y", "s_out"], ["x", "s_in", "w", "b"], [("y", "x"), ("s_out", "s_in")]), ids=str)
def test_short_conv_decode(lib, case):
    assert refused(lib.short_conv_decode, CTOK_ORDER, dict(CTOK, act=1, dt=0, N=N, C=C, W=W, stream=None),
                   shift(CTOK, case))


NORM = arrays("x res w b y sum")
NORM_ORDER = "x res w b eps dt rows D y sum stream".split()


@pytest.mark.parametrize("case", cases(["y", "sum"], ["x", "res", "w", "b"],
                                       [(o, i) for o in ("y", "sum") for i in ("x", "res")]), ids=str)
def test_layer_norm_fwd(lib, case):
    assert refused(lib.layer_norm_fwd, NORM_ORDER, dict(NORM, eps=1e-5, dt=0, rows=T, D=C, stream=None), shift(NORM, case))


NBWD = arrays("sum w dy ds dx dw db ws")
NBWD_ORDER = "sum w eps dt rows D dy ds dx dw db ws wsb stream".split()


@pytest.mark.parametrize("case", cases(["dx", "dw", "db"], ["sum", "dy", "ds", "w"],
                                       [("dx", "sum"), ("dx", "dy"), ("dx", "ds")]), ids=str)
def test_layer_norm_bwd(lib, case):
    assert refused(lib.layer_norm_bwd, NBWD_ORDER, dict(NBWD, eps=1e-5, dt=0, rows=T, D=C, wsb=BIG, stream=None),
                   shift(NBWD, case))


@pytest.mark.parametrize("i", [n for n in NBWD if n != "ws"])
def test_layer_norm_bwd_workspace(lib, i):
    assert refused(lib.layer_norm_bwd, NBWD_ORDER, dict(NBWD, eps=1e-5, dt=0, rows=T, D=C, wsb=BIG, stream=None),
                   dict(ws=NBWD[i]))
