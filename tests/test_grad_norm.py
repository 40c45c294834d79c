"""grad_norm and clip_grad_norm against float64.

Tolerances: a thread adds up at most 66 squares in fp32, in two chains, the rest is fp64: 35 2^-24 of the sum, half of that of the
norm, and its rounding to fp32.  A scaled value is off by the norm's error and two roundings, then half a step of its type.
"""
import math

import pytest
import torch

import row_wise_online_gb300 as rwo
from train_util import BF, F32, FP, TYPES, U, assert_close, half_step

pytestmark = pytest.mark.gpu
NORM = 22 * U


@pytest.fixture(scope="module", autouse=True)
def _built():
    from row_wise_online_gb300 import _build

    _build.build()
    torch.cuda.set_device(0)


def make(sizes, dts, seed=0, sd=0.1):
    gen = torch.Generator().manual_seed(seed)
    return [(sd * (1 + k % 3) * torch.randn(n, generator=gen)).to(dts[k % len(dts)]) for k, n in enumerate(sizes)]


def norm64(ts, scale=1.0):
    scale = float(torch.tensor(scale, dtype=F32))
    return abs(scale) * math.sqrt(sum(float(t.double().pow(2).sum()) for t in ts))


def check(cpu, gpu, max_norm, out=None, scale=1.0):
    norm = norm64(cpu, scale)
    limit = float(torch.tensor(max_norm, dtype=F32))
    before = [t.clone() for t in gpu]
    got = rwo.clip_grad_norm(gpu, max_norm, out=out, scale=scale)
    assert rwo.get_status() == rwo.OK and got.shape == () and abs(float(got) - norm) <= NORM * norm
    alone = rwo.grad_norm(before, scale=scale)
    assert torch.equal(got, alone)
    k = float(torch.tensor(scale, dtype=F32)) * (min(1.0, limit / norm) if norm > 0 else 1.0)
    for t, o in zip(cpu, gpu if out is None else out):
        ref = t.double() * k
        assert_close(o, ref.view(o.shape), ((NORM + 3 * U) * ref.abs() + half_step(ref, o.dtype)).view(o.shape))
    if out is not None:
        assert all(torch.equal(a, b) for a, b in zip(before, gpu))
    return got


SIZES = [[1], [0, 3], [7, 8, 9], [4096], [4097, 8191, 8192, 8193], [16384, 1, 0, 5, 100003], [1 << 20, (1 << 20) + 1], [33] * 70]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("dts", [[F32], [BF], [FP], [BF, F32, FP]])
@pytest.mark.parametrize("factor", [0.3, 2.0])
def test_lists(sizes, dts, factor):
    """Clipped and not, in place, into tensors of their own types and into fp32."""
    cpu = make(sizes, dts)
    limit = factor * norm64(cpu)
    for scale in (1.0, 0.125):
        check(cpu, [t.cuda() for t in cpu], limit * scale, scale=scale)
    check(cpu, [t.cuda() for t in cpu], limit, out=[torch.full_like(t, math.nan).cuda() for t in cpu])
    check(cpu, [t.cuda() for t in cpu], 3 * limit, out=[torch.full(t.shape, math.nan, device="cuda") for t in cpu], scale=-3.0)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("lead", range(8))
def test_views_of_a_bucket(dt, lead):
    """Tensors side by side in one buffer, at every alignment; what lies beside them stays."""
    sizes = [1, 2, 3, 5, 17, 4099, 8200, 12289, 8192 + 7]
    cpu = make(sizes, [dt], 1)
    flat = torch.full((lead + sum(sizes) + 9,), math.inf, dtype=dt, device="cuda")
    for out_dt in {dt, F32}:
        views = list(flat[lead: lead + sum(sizes)].split(sizes))
        for v, t in zip(views, cpu):
            v.copy_(t)
        for out_lead in (lead, 0, 3):
            target = torch.full((out_lead + sum(sizes) + 5,), math.inf, dtype=out_dt, device="cuda")
            check(cpu, views, 0.5 * norm64(cpu), out=list(target[out_lead: out_lead + sum(sizes)].split(sizes)))
            assert int(torch.isinf(target).sum()) == out_lead + 5
    check(cpu, views, 0.5 * norm64(cpu))
    assert int(torch.isinf(flat).sum()) == lead + 9


@pytest.mark.parametrize("count", [63, 64, 65, 511, 512, 513, 1500])
def test_many_tensors(count):
    sizes = [(k * 37) % 300 for k in range(count)]
    cpu = make(sizes, [BF, F32], 2)
    check(cpu, [t.cuda() for t in cpu], 0.1 * norm64(cpu))


def test_shapes_and_empty():
    a = torch.randn(3, 5, 7, device="cuda")
    b = torch.randn(2, device="cuda")
    want = math.sqrt(float(a.double().pow(2).sum() + b.double().pow(2).sum()))
    assert abs(float(rwo.grad_norm([a, b])) - want) <= NORM * want
    assert float(rwo.grad_norm([])) == 0 and float(rwo.clip_grad_norm([], 1.0)) == 0
    z = torch.zeros(100, device="cuda")
    assert float(rwo.clip_grad_norm([z], 1.0)) == 0 and not z.any()
    out = torch.empty((), device="cuda")
    assert rwo.grad_norm([a], norm_out=out) is out
    assert float(rwo.grad_norm(iter([a, b]), scale=0.0)) == 0


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("power", [-130, -120, -64, -50, -46, 40, 59, 61, 63, 100, 120])
def test_magnitudes(dt, power):
    """Squares far outside fp32's range; the sum itself is not."""
    cpu = [(torch.randn(n, generator=torch.Generator().manual_seed(n)).clamp(-3, 3).double() * 2.0 ** power).to(dt) for n in (1, 100, 20000)]
    got, want = float(rwo.grad_norm([t.cuda() for t in cpu])), norm64(cpu)
    assert abs(got - want) <= (NORM + U) * want + 2.0 ** -149
    mixed = cpu + [torch.ones(5, dtype=dt)]
    assert abs(float(rwo.grad_norm([t.cuda() for t in mixed])) - norm64(mixed)) <= (NORM + U) * norm64(mixed)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("dt", TYPES)
def test_not_finite(bad, dt):
    """An infinity or NaN shows in the norm; nothing is limited, in place nothing is touched."""
    cpu = make([5000, 40], [dt], 3)
    cpu[0][4321] = bad
    gpu = [t.cuda() for t in cpu]
    norm = rwo.clip_grad_norm(gpu, 0.01)
    assert (math.isnan(float(norm)) if math.isnan(bad) else float(norm) == math.inf)
    assert all(torch.equal(a.cpu().nan_to_num(nan=9), b.nan_to_num(nan=9)) for a, b in zip(gpu, cpu))
    out = [torch.empty_like(t) for t in gpu]
    rwo.clip_grad_norm(gpu, 0.01, out=out, scale=0.5)
    assert torch.equal(out[1].cpu(), (cpu[1].float() * 0.5).to(dt))


def test_norm_above_fp32():
    t = torch.full((64,), 3e38, device="cuda")
    assert float(rwo.clip_grad_norm([t], 1.0)) == math.inf and (t == t[0]).all() and float(t[0]) == float(torch.tensor(3e38))


def test_repeats_streams_and_graphs():
    cpu = make([100000, 33, 70000], [BF, F32], 4)
    gpu = [t.cuda() for t in cpu]
    out = [torch.empty_like(t) for t in gpu]
    want = rwo.clip_grad_norm(gpu, 1.0, out=out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out2 = [torch.empty_like(t) for t in gpu]
    got = rwo.clip_grad_norm(gpu, 1.0, out=out2, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and all(torch.equal(a, b) for a, b in zip(out, out2))
    ws, norm = rwo.grad_norm_workspace(3), torch.zeros((), device="cuda")
    held = [torch.zeros_like(t) for t in gpu]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rwo.clip_grad_norm(held, 1.0, norm_out=norm, workspace=ws)
    for _ in range(2):
        for a, b in zip(held, gpu):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, want) and all(torch.equal(a, b) for a, b in zip(out, held))


def test_a_tensor_listed_twice():
    a, b = (t.cuda() for t in make([100, 300], [F32]))
    e = a[:0]
    assert abs(float(rwo.grad_norm([a, a])) - float(a.double().pow(2).sum() * 2) ** 0.5) <= NORM * float(a.double().norm()) * 2 ** 0.5
    keep = a.clone()
    for call in (lambda: rwo.clip_grad_norm([a, b, a], 1.0), lambda: rwo.clip_grad_norm([a, a], 1.0, out=[keep, keep])):
        with pytest.raises(ValueError, match="twice"):
            call()
    assert torch.equal(a, keep)
    rwo.clip_grad_norm([a, e, e, b], 1.0)  # empty ones may come again
    assert rwo.get_status() == rwo.OK
