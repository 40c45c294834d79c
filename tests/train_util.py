"""Shared by the tests of the training step: element types, half steps, rows at odd places."""
import torch

F32, BF, FP = torch.float32, torch.bfloat16, torch.float16
TYPES = [F32, BF, FP]
U = 2.0 ** -24  # half a step of fp32, relative


def half_step(ref, dt):
    """Half a step of the element type around values ``ref`` (fp64): relative for normal values, absolute below them."""
    info = torch.finfo(dt)
    return torch.clamp(ref.abs(), min=float(info.tiny)) * (info.eps / 2)


def placed(t, shift=0, pad=0):
    """A CUDA copy of a matrix whose first element lies ``shift`` elements behind a 16-byte boundary and whose rows
    are ``pad`` elements further apart than their length; the gaps hold NaN."""
    M, N = t.shape
    buf = torch.full((shift + M * (N + pad) + 64,), float("nan"), dtype=t.dtype, device="cuda")
    view = buf[shift: shift + M * (N + pad)].view(M, N + pad)[:, :N]
    view.copy_(t)
    return view


def assert_close(got, ref, tol, what=""):
    """Every element within its own tolerance; what is not finite in the reference has to be the same."""
    got, ref, tol = got.detach().double().cpu(), ref.double().cpu(), torch.as_tensor(tol, dtype=torch.float64).cpu().expand_as(ref)
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN at other places"
    inf = ~fine & ~torch.isnan(ref)
    assert torch.equal(got[inf], ref[inf]), f"{what}: infinities differ"
    off = (got - ref).abs()[fine] - tol[fine]
    assert off.numel() == 0 or off.max() <= 0, f"{what}: off by {off.max():.3g} more than the tolerance at {int((off > 0).sum())} of {off.numel()}"
