"""la_* and gated_norm_* on the host: every refusal comes before any HIP call
(fake pointers, no device), and the wrappers refuse what the kernels do not do."""
import ctypes

import pytest
import torch

import chunked_gated_delta_kda_amd as kda

FAKE = ctypes.c_void_p(0x1000)
odd = lambda n: ctypes.c_void_p(0x1000 + n)  # noqa: E731


@pytest.fixture(scope="module")
def lib():
    return kda.load()


def la_fwd(lib, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, ld=FAKE, scale=0.1, h0=None, hT=None, cu=None, N=1, B=1, T=16, H=1, K=128,
             V=128, o=FAKE, ws=None, wsb=0, seg=0, stream=None)
    assert set(over) <= set(a)
    return lib.la_fwd(*{**a, **over}.values())


COMMON = [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(ld=None), 1), (dict(B=0), 1), (dict(T=-1), 1),
    (dict(H=0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(K=96), 2), (dict(V=256), 2),
    (dict(cu=FAKE, B=2, N=2), 1), (dict(cu=FAKE, N=0), 1), (dict(cu=odd(2)), 1), (dict(B=1 << 16, T=1 << 15), 1),
    (dict(q=odd(8)), 1), (dict(k=odd(2)), 1), (dict(v=odd(8)), 1), (dict(h0=odd(8)), 1), (dict(ld=odd(2)), 1),
    # segments need the workspace of their states
    (dict(T=1024, seg=4), 3), (dict(T=1024, seg=4, ws=FAKE, wsb=1000), 3),
    (dict(T=1024, seg=4, ws=odd(16), wsb=1 << 30), 3),
    # more (slot, head) pairs than a grid addresses
    (dict(cu=FAKE, N=1 << 24, H=4), 1), (dict(B=1 << 20, T=1024, H=64, seg=1, ws=FAKE, wsb=1 << 62), 1),
]


@pytest.mark.parametrize("over,code", COMMON + [(dict(o=None), 1), (dict(o=odd(8)), 1), (dict(hT=odd(4)), 1)])
def test_la_fwd_rejects_on_host(lib, over, code):
    assert la_fwd(lib, **over) == code


def la_bwd(lib, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, ld=FAKE, scale=0.1, h0=None, cu=None, N=1, B=1, T=16, H=1, K=128, V=128, do=FAKE,
             dfin=None, dq=FAKE, dk=FAKE, dv=FAKE, dh0=None, ws=None, wsb=0, seg=0, stream=None)
    assert set(over) <= set(a)
    return lib.la_bwd(*{**a, **over}.values())


@pytest.mark.parametrize("over,code", COMMON + [
    (dict(do=None), 1), (dict(dq=None), 1), (dict(dk=None), 1), (dict(dv=None), 1), (dict(do=odd(8)), 1),
    (dict(dq=odd(2)), 1), (dict(dk=odd(8)), 1), (dict(dv=odd(8)), 1), (dict(dfin=odd(8)), 1), (dict(dh0=odd(4)), 1)])
def test_la_bwd_rejects_on_host(lib, over, code):
    assert la_bwd(lib, **over) == code


def test_la_workspace_holds_the_segments_states(lib):
    assert kda.la_workspace_size(2, 2048, 32, 128, 128, segment_chunks=-1) == 256  # no segments, none needed
    assert kda.la_workspace_size(1, 100, 1, 96, 128) == 0
    assert kda.la_workspace_size(0, 100, 1, 128, 128) == 0
    assert kda.la_workspace_size(1, 100, 1, 128, 128, num_seqs=0) == 0
    state = 3 * 128 * 64 * 4
    # 2 sequences x 4 segments of 4 chunks
    assert kda.la_workspace_size(2, 1000, 3, 128, 64, segment_chunks=4) == 8 * state
    # packed: at most total / length + one a sequence
    assert kda.la_workspace_size(1, 1000, 3, 128, 64, num_seqs=5, segment_chunks=4) == 8 * state
    assert kda.la_workspace_size(1, 1000, 3, 128, 64, num_seqs=5, segment_chunks=4, backward=True) == 16 * state
    # a segment as long as the batch is the whole sequence
    assert kda.la_workspace_size(1, 1024, 3, 128, 64, segment_chunks=16) == 256


def la_decode(lib, **over):
    a = dict(q=FAKE, k=FAKE, v=FAKE, ld=FAKE, scale=0.1, s_in=None, s_out=FAKE, N=2, H=4, K=128, V=128, o=FAKE,
             stream=None)
    assert set(over) <= set(a)
    return lib.la_decode(*{**a, **over}.values())


@pytest.mark.parametrize("over,code", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(ld=None), 1), (dict(s_out=None), 1),
    (dict(o=None), 1), (dict(N=0), 1), (dict(H=0), 1), (dict(scale=float("nan")), 1), (dict(K=32), 2),
    (dict(V=96), 2), (dict(q=odd(8)), 1), (dict(k=odd(8)), 1), (dict(v=odd(4)), 1), (dict(o=odd(4)), 1),
    (dict(s_in=odd(4)), 1), (dict(s_out=odd(8)), 1), (dict(N=1 << 20, H=1 << 11), 1)])
def test_la_decode_rejects_on_host(lib, over, code):
    assert la_decode(lib, **over) == code


def norm_fwd(lib, **over):
    a = dict(x=FAKE, gate=FAKE, w=FAKE, res=None, rs=None, act=0, eps=1e-6, tokens=4, H=2, D=128, y=FAKE, stream=None)
    assert set(over) <= set(a)
    return lib.gated_norm_fwd(*{**a, **over}.values())


NORM = [
    (dict(x=None), 1), (dict(w=None), 1), (dict(act=2), 1), (dict(act=-1), 1), (dict(eps=-1e-6), 1),
    (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1), (dict(tokens=-1), 1), (dict(H=0), 1), (dict(D=0), 1),
    (dict(D=100), 2), (dict(D=520), 2), (dict(D=4), 2), (dict(tokens=1 << 30, H=2), 1), (dict(res=FAKE), 1),
    (dict(rs=FAKE), 1), (dict(x=odd(8)), 1), (dict(gate=odd(8)), 1), (dict(res=odd(8), rs=FAKE), 1),
    (dict(w=odd(2)), 1), (dict(res=FAKE, rs=odd(2)), 1)]


@pytest.mark.parametrize("over,code", NORM + [(dict(y=None), 1), (dict(y=odd(8)), 1)])
def test_gated_norm_fwd_rejects_on_host(lib, over, code):
    assert norm_fwd(lib, **over) == code


def norm_bwd(lib, **over):
    a = dict(x=FAKE, gate=FAKE, w=FAKE, res=None, rs=None, act=0, eps=1e-6, tokens=4, H=2, D=128, dy=FAKE, dx=FAKE,
             dgate=FAKE, dw=FAKE, dres=None, drs=None, ws=FAKE, wsb=1 << 30, stream=None)
    assert set(over) <= set(a)
    return lib.gated_norm_bwd(*{**a, **over}.values())


@pytest.mark.parametrize("over,code", NORM + [
    (dict(dy=None), 1), (dict(dx=None), 1), (dict(dgate=None), 1), (dict(dw=None), 1), (dict(dy=odd(8)), 1),
    (dict(res=FAKE, rs=FAKE, drs=FAKE), 1), (dict(res=FAKE, rs=FAKE, dres=FAKE), 1), (dict(ws=None), 3),
    (dict(wsb=64), 3), (dict(ws=odd(16)), 3), (dict(dx=odd(8)), 1), (dict(dgate=odd(8)), 1), (dict(dw=odd(2)), 1)])
def test_gated_norm_bwd_rejects_on_host(lib, over, code):
    assert norm_bwd(lib, **over) == code


def test_norm_without_tokens_needs_no_rows(lib):
    assert norm_fwd(lib, tokens=0, x=None, gate=None, y=None) == 0  # nothing enqueued
    assert lib.gated_norm_bwd_workspace_size(0, 2, 128) > 0
    assert lib.gated_norm_bwd_workspace_size(4, 2, 100) == 0


def test_wrappers_refuse():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    q, ld = bf(1, 4, 2, 64), torch.zeros(2)
    with pytest.raises(NotImplementedError, match="log_decay"):
        kda.chunk_la(q, q, q, ld.clone().requires_grad_())
    with pytest.raises(ValueError, match="GPU"):
        kda.chunk_la(q, q, q, ld)
    with pytest.raises(ValueError, match="GPU"):
        kda.la_decode(q[0], q[0], q[0], ld)
    with pytest.raises(TypeError):
        kda.la_fwd(q.float(), q, q, ld)
    with pytest.raises(ValueError, match="GPU"):
        kda.gated_norm(q, q, torch.ones(64))


def test_la_refuses_rows_that_32_bit_offsets_do_not_reach(lib):
    """A chunk's rows are addressed by 32-bit byte offsets: at most 65536 heads."""
    assert la_fwd(lib, H=65537) == 1
    assert la_bwd(lib, H=65537) == 1


def test_la_workspace_of_unsupported_heads(lib):
    assert kda.la_workspace_size(1, 16, 65537, 64, 64) == 0
    assert kda.la_workspace_size(1, 16, 65537, 64, 64, backward=True) == 0


@pytest.mark.parametrize("packed,N,T,H,seg,refused", [
    (False, 1 << 23, 2, 64, 0, True), (False, 1 << 23, 2, 4, -1, True), (False, 1 << 23, 2, 3, 0, False),
    (False, 1 << 20, 1024, 64, 1, True), (False, 1 << 19, 1024, 4, 4, False), (False, 1 << 25, 1, 1, 0, True),
    (False, (1 << 25) - 1, 1, 1, 0, False), (False, 3, 1 << 20, 2048, 1, True), (False, 3, 1 << 20, 512, 1, False),
    (True, 1 << 24, 5, 2, 0, True), (True, (1 << 24) - 1, 5, 2, 0, False), (True, 7, (1 << 31) - 1, 1, 1, True),
    (True, 7, 1 << 30, 1, 1, False)])
def test_la_workspace_size_is_0_where_the_call_refuses(lib, packed, N, T, H, seg, refused):
    """More pairs of a head and a slot than a launch counts: refused by the size already,
    not by an allocation of terabytes."""
    B = 1 if packed else N
    over = dict(cu=FAKE if packed else None, N=N, B=B, T=T, H=H, K=64, V=64, seg=seg)
    for call, backward in ((la_fwd, False), (la_bwd, True)):
        size = kda.la_workspace_size(B, T, H, 64, 64, N, seg, backward=backward)
        assert (size == 0) == refused
        if refused:  # (of a call that is not, nothing may be enqueued here)
            assert call(lib, **over, ws=FAKE, wsb=1 << 62) == 1
        elif size > 256:
            assert call(lib, **over) == 3


def test_workspaces_that_are_not_one_piece_are_refused():
    """The kernels write a workspace from its address on: an expanded or strided view
    has as many elements, but not the memory."""
    from chunked_gated_delta_kda_amd import _binding as b

    cpu = torch.device("cpu")
    piece = torch.empty(4096, dtype=torch.uint8)
    b._need_workspace(piece, 4096, cpu)
    b._need_workspace(piece.view(64, 64)[:], 4096, cpu)
    with pytest.raises(kda.LibKdaError, match="WORKSPACE"):
        b._need_workspace(piece, 4097, cpu)
    with pytest.raises(ValueError, match="contiguous"):
        b._need_workspace(piece[:1].expand(4096), 4096, cpu)
    with pytest.raises(ValueError, match="contiguous"):
        b._need_workspace(torch.empty(8192, dtype=torch.uint8)[::2], 4096, cpu)
