"""The factor of clip_grad_norm: held in more bits than fp32, and the product rounded once.

The gradients here have norms without rounding (bf16 values of one power of 2: 33 of their squares add up to less than 24 bits, and
sums in fp64 are exact), so that what comes back is off by half a step of its type and no more.  Half a step of fp32 is 2^-24 of the value; 1.0001
of it allows for the 2^-48 that hi + lo leaves and for the square root in fp64.
"""
import math

import pytest
import torch

import row_wise_online_gb300 as rwo
from train_util import BF, F32, FP, U, assert_close, half_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from row_wise_online_gb300 import _build

    _build.build()
    torch.cuda.set_device(0)


def grads(sizes, power=0, seed=1):
    """bf16 values of 2^power to 2^(power + 1) and either sign."""
    gen = torch.Generator().manual_seed(seed)
    out = []
    for n in sizes:
        m = torch.randint(128, 256, (n,), generator=gen).double() / 128
        out.append((torch.where(torch.rand(n, generator=gen) < 0.5, -m, m) * 2.0 ** power).to(BF))
    return out


def norm64(ts):
    return math.sqrt(math.fsum(float(t.double().pow(2).sum()) for t in ts))


SIZES = [[5000], [7, 4097, 8192], [200000, 33, 70001], [129] * 70]  # one launch for all, and two


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("limit", [0.1, 1 + 2.0 ** -24, 1 / 3, math.pi])
@pytest.mark.parametrize("scale", [1.0, -0.125])
def test_rounded_once(sizes, limit, scale):
    cpu = grads(sizes)
    k = scale * limit / (abs(scale) * norm64(cpu))
    for source in (BF, F32):
        gpu = [t.to(source).cuda() for t in cpu]
        out = [torch.empty(t.shape, device="cuda") for t in cpu]
        rwo.clip_grad_norm(gpu, limit, out=out, scale=scale)
        assert rwo.get_status() == rwo.OK
        for t, o in zip(cpu, out):
            ref = t.double() * k
            assert_close(o, ref, 1.0001 * U * ref.abs())
    rwo.clip_grad_norm(gpu, limit, scale=scale)  # fp32 in place: the same
    assert all(torch.equal(a, b) for a, b in zip(gpu, out))


@pytest.mark.parametrize("power,limit", [(110, 1.0), (118, 1e-3), (118, 1.0), (118, 1e-30), (60, 1e-38), (30, 1e-30)])
def test_factors_below_fp32(power, limit):
    """A norm near fp32's largest limited to an ordinary one, and further: what comes back is a normal number or nearly."""
    cpu = grads([60, 5000, 8192], power)
    norm = norm64(cpu)
    assert norm <= 3.4e38
    out = [torch.empty(t.shape, device="cuda") for t in cpu]
    got = rwo.clip_grad_norm([t.cuda() for t in cpu], limit, out=out)
    assert abs(float(got) - norm) <= 1.0001 * U * norm
    for t, o in zip(cpu, out):
        ref = t.double() * (limit / norm)
        # below fp32's normal values half a step is 2^-150, twice: of the smaller part, and of the result
        assert_close(o, ref, 1.0001 * U * ref.abs() + torch.where(ref.abs() < 2.0 ** -100, 2.0 ** -149, 0.0))


@pytest.mark.parametrize("dt", [BF, FP])
def test_own_types(dt):
    cpu = [t.to(dt) for t in grads([5000, 33])]
    gpu = [t.cuda() for t in cpu]
    rwo.clip_grad_norm(gpu, 0.7)
    for t, o in zip(cpu, gpu):
        ref = t.double() * (0.7 / norm64(cpu))
        assert_close(o, ref, 1.0001 * U * ref.abs() + half_step(ref, dt))


def test_infinities_are_kept():
    """Where the norm is not finite the scale alone is applied, an infinity stays one whatever the scale's digits."""
    for scale in (1 / 3, 0.1, -7.3):
        t = torch.tensor([math.inf, -math.inf, 1.0, 0.0], device="cuda")
        out = [torch.empty_like(t)]
        assert float(rwo.clip_grad_norm([t], 0.5, out=out, scale=scale)) == math.inf
        assert torch.equal(out[0], t * torch.tensor(scale, dtype=F32))


def test_the_limit_in_64_bits():
    """Limits outside fp32's range are taken as they are: one limits to almost nothing, one limits nothing."""
    t = torch.full((4,), 2.0 ** 100, device="cuda")
    out = [torch.empty_like(t)]
    rwo.clip_grad_norm([t], 1e-50, out=out)  # 0.5e-50: below fp32's least
    assert not out[0].any()
    rwo.clip_grad_norm([t], 1e60, out=out)
    assert torch.equal(out[0], t)
