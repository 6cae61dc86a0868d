"""Helpers shared by the GPU tests of the operators around a block."""
import torch

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def to_gpu(d):
    return {k: t.to(DEV) if isinstance(t, torch.Tensor) else t for k, t in d.items()}


def near(name, got, want_and_bound):
    """Within the bound of the arithmetic and half a step of the output's type.  What lies
    below the type's normal numbers (and gates below 2^-126, which count as zero) may be
    lost: 2^-120 is far above it and far below any value here."""
    want, bound = want_and_bound
    g = got.detach().double().cpu()
    assert g.shape == want.shape, (name, g.shape, want.shape)
    if not g.numel():
        return
    assert torch.isfinite(g).all(), name
    half = torch.finfo(got.dtype).eps / 2
    over = (g - want).abs() - bound - half * (want.abs() + bound) - 2.0 ** -120
    assert over.max() <= 0, (name, over.max().item(), (g - want).abs().max().item())


def offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32)
