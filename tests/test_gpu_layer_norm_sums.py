"""The layer norm's sums over very many rows (dweight and dbias), at the same tolerance as
over a few: 2^-17 of the absolute terms, and what the rows' own norm may be off by.

The rows are three, over and over, so that roundings of a running sum in fp32 do not cancel
(2048 additions of one number are off by up to 2^-13 of the sum), and the sums in 64 bits
are those of three rows."""
import pytest
import torch

import chunked_gated_delta_kda_amd as kda
from block_util import DEV, TYPES, near
from oracle import block as ref
from parity_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def give_memory_back():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("rows,D,dtype", [
    (1 << 20, 1024, "fp32"), ((1 << 20) + 3, 1000, "bf16"), ((1 << 18) + 5, 4096, "bf16"), ((1 << 18) + 7, 4104, "fp32"),
    ((1 << 17) + 1, 8192, "bf16"), (70001, 16384, "bf16"), (50003, 16384, "fp32"), ((1 << 22) + 9, 8, "fp32"),
    ((1 << 21) + 33, 64, "bf16"), ((1 << 21) + 1, 136, "fp32"), ((1 << 20) + 1, 512, "bf16")])
def test_sums_over_many_rows(rows, D, dtype):
    gen = torch.Generator().manual_seed(D)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    tt = TYPES[dtype]
    x, w, b = n(3, D).to(tt), 1 + n(D) / 8, n(D)
    dy = (0.1 + 0.6 * torch.rand(3, D, generator=gen)).to(tt)
    count = torch.tensor([len(range(r, rows, 3)) for r in range(3)], dtype=torch.float64)
    value, bound = {}, {}
    for r in range(3):
        one = ref.layer_norm_all(x[r:r + 1], w, b, 1e-5, dy[r:r + 1])
        for k in ("dweight", "dbias"):
            value[k] = value.get(k, 0) + count[r] * one[k][0]
            bound[k] = bound.get(k, 0) + count[r] * one[k][1]
    say(f"[layer norm] {rows} rows of {D} {dtype}")
    at = torch.arange(rows, device=DEV) % 3
    many = [t.to(DEV)[at] for t in (x, dy)]
    r = kda.layer_norm_bwd(many[0], w.to(DEV), many[1])
    for k in ("dweight", "dbias"):
        near(k, r[k], (value[k], bound[k]))
    few = kda.layer_norm_bwd(many[0][:300], w.to(DEV), many[1][:300])
    assert torch.equal(r["dx"][:300], few["dx"]) and torch.equal(r["dx"][-100:], few["dx"][[(rows - 100 + i) % 3 for i in range(100)]])


@pytest.mark.parametrize("dtype,D", [("fp32", 1024), ("bf16", 4096), ("bf16", 16384)])
def test_a_workspace_that_is_given_serves_many_rows(dtype, D):
    """Its size is the one that is asked for, whatever it holds, and what is behind it stays."""
    rows = 40000
    gen = torch.Generator(device=DEV).manual_seed(5)
    x, dy = (torch.randn(rows, D, generator=gen, device=DEV).to(TYPES[dtype]) for _ in range(2))
    w = torch.randn(D, generator=gen, device=DEV)
    need = kda.load().layer_norm_bwd_workspace_size(int(dtype == "fp32"), rows, D)
    want = kda.layer_norm_bwd(x, w, dy)
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device=DEV)
    got = kda.layer_norm_bwd(x, w, dy, workspace=ws[:need])
    assert all(torch.equal(got[k], want[k]) for k in want) and bool((ws[need:] == 255).all())
