"""cross_entropy_rows_grad against float64.

Tolerances: the softmax is within 1e-5 of itself (the library's bound), so are 1 + 2 z LSE and the product with w; the
label's and the smoothing's terms are two fp32 products and a subtraction: 4 2^-24 of what is subtracted.  Then half a step of the
element type, and 2^-126 of the factor, where the hardware exponential flushes.  Loss and LSE: 1e-5 max(1, |terms|).
"""
import math

import pytest
import torch

import row_wise_online_gb300 as rwo
from train_util import BF, F32, FP, TYPES, U, assert_close, half_step, placed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from row_wise_online_gb300 import _build

    _build.build()
    torch.cuda.set_device(0)


def reference(x, labels, upstream=None, grad_scale=1.0, eps=0.0, z=0.0):
    """loss, lse, grad and the gradient's tolerance before rounding, in 64 bits on the CPU."""
    x = x.double().cpu()
    labels = labels.cpu()
    M, N = x.shape
    live, bad = labels >= 0, labels >= N
    t = labels.clamp(0, N - 1)[:, None]
    m = x.amax(1, keepdim=True)
    empty = torch.isinf(m) & (m < 0)
    # relative to the maximum: at |x| = 1e30 even 64 bits lose ln d beside m (N equal entries have the loss ln N)
    log_d = torch.where(empty, -math.inf, torch.logsumexp(x - m, 1, keepdim=True))
    lse = m + log_d
    loss = (1 - eps) * (log_d + (m - x.gather(1, t))) + z * lse ** 2
    if eps:
        loss = loss + eps * (log_d + (m - x)).mean(1, keepdim=True)
    loss = torch.where(empty | bad[:, None], math.nan, loss)
    w = torch.full((M, 1), float(torch.tensor(grad_scale, dtype=F32)), dtype=torch.float64)
    if upstream is not None:
        w = w * upstream.double().cpu()[:, None]
    p = torch.where(empty, math.nan, (x - m - log_d).exp())
    first = w * p * (1 + 2 * z * lse)
    grad = first - w * eps / N
    grad = grad.scatter_add(1, t, -(1 - eps) * w)
    grad = torch.where(bad[:, None], math.nan, grad)
    dead = ~live[:, None]
    tol = 1e-5 * first.abs() + 4 * U * w.abs() * eps / N + 2.0 ** -126 * (1 + w.abs())
    tol = tol.scatter_add(1, t, 4 * U * (1 - eps) * w.abs())
    return torch.where(dead, 0.0, loss)[:, 0], lse[:, 0], torch.where(dead, 0.0, grad), torch.where(dead, 0.0, tol)


def check(x, labels, grad=None, pitched=None, **kw):
    """Calls with kw (grad_scale, upstream, eps, z) and compares; returns what came back."""
    M, N = x.shape
    loss_ref, lse_ref, grad_ref, tol = reference(x, labels, kw.get("upstream"), kw.get("grad_scale", 1.0), kw.get("eps", 0.0), kw.get("z", 0.0))
    lse = torch.full((M,), math.nan, device="cuda")
    loss, g = rwo.cross_entropy_rows_grad(x, labels, grad=grad, lse_out=lse, upstream=kw.get("upstream"), grad_scale=kw.get("grad_scale", 1.0),
                                          label_smoothing=kw.get("eps", 0.0), z_loss=kw.get("z", 0.0))
    status = rwo.get_status()
    assert status == (rwo.ERR_INVALID_ARG if bool((labels >= N).any()) else rwo.OK)
    size = torch.where(torch.isfinite(loss_ref), loss_ref.abs(), torch.zeros(())).clamp(min=1) + torch.where(torch.isfinite(lse_ref), kw.get("z", 0.0) * lse_ref ** 2, torch.zeros(()))
    assert_close(loss, loss_ref, 1e-5 * size, "loss")
    assert_close(lse, lse_ref, 1e-5 * torch.where(torch.isfinite(lse_ref), lse_ref.abs(), torch.zeros(())).clamp(min=1), "lse")
    assert_close(g, grad_ref, tol + half_step(grad_ref, x.dtype), "grad")
    return loss, lse, g


def logits(M, N, dt, seed=0, sd=3.0):
    gen = torch.Generator().manual_seed(seed * 1000 + N)
    x = (sd * torch.randn(M, N, generator=gen)).to(dt)
    labels = torch.randint(0, N, (M,), generator=gen)
    labels[torch.rand(M, generator=gen) < 0.2] = -100
    return x, labels.cuda()


LENGTHS = [1, 2, 3, 7, 8, 31, 64, 100, 129, 1000, 1024, 4096, 5003, 8192, 16384, 16385, 32000, 32768, 50021, 65536, 100001, 131072, 262144]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("N", LENGTHS)
def test_lengths(N, dt):
    M = 5 if N > 60000 else 37
    x, labels = logits(M, N, dt)
    check(x.cuda(), labels, grad_scale=1.0 / M)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("N", [1, 5, 777, 4096, 20000, 50021, 131072, 300000])
def test_smoothing_z_and_weights(N, dt):
    M = 7
    x, labels = logits(M, N, dt, 1)
    w = torch.rand(M, generator=torch.Generator().manual_seed(5)).cuda()
    check(x.cuda(), labels, upstream=w, grad_scale=3.0, eps=0.1, z=1e-3)
    check(x.cuda(), labels, eps=0.3)
    check(x.cuda(), labels, z=1e-2)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("N", [96, 1000, 4096, 32003, 131072])
@pytest.mark.parametrize("shift,pad", [(0, 8), (0, 7), (1, 0), (3, 5), (4, 24)])
def test_pitches_and_offsets(N, dt, shift, pad):
    """Rows that start anywhere, x and the gradient at the same offset within 16 bytes or at others."""
    x, labels = logits(9, N, dt, 2)
    xp = placed(x, shift, pad)
    check(xp, labels)
    gbuf = placed(torch.zeros_like(x), shift, pad)
    _, _, a = check(xp, labels, grad=gbuf)
    check(xp, labels, grad=placed(torch.zeros_like(x), (shift + 1) % 8, pad + 2))
    # in place: the logits become their gradient, the gaps stay
    base = xp._base if xp._base is not None else xp
    kept = torch.isnan(base).sum()
    rwo.cross_entropy_rows_grad(xp, labels, grad=xp)
    assert torch.equal(a, xp) and torch.isnan(base).sum() == kept


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("N", [40, 4096, 33000, 131072])
@pytest.mark.parametrize("eps", [0.0, 0.1])
def test_masked_entries(N, dt, eps):
    """-inf among the logits: parts of rows, the label, all but the label, all; ignored rows may hold anything."""
    x, labels = logits(8, N, dt, 3)
    labels[:] = torch.arange(8) % N
    x[0, N // 2:] = -math.inf
    x[1, 1] = -math.inf          # its label
    x[2, :] = -math.inf
    x[2, 2] = 1.5                # all but its label
    x[3, :] = -math.inf          # nothing left
    x[4, : N // 2] = -math.inf
    x[4, 4] = 0.5
    x[5, :] = math.nan
    labels[5] = -1
    x[6, :] = -math.inf
    labels[6] = -7
    x[7, 0] = -math.inf
    keep = [0, 1, 2, 3, 4, 6, 7]
    lse = torch.empty(8, device="cuda")
    loss, g = rwo.cross_entropy_rows_grad(x.cuda(), labels, lse_out=lse, label_smoothing=eps)
    assert loss[5] == 0 and not g[5].any() and torch.isnan(lse[5])
    check(x[keep].cuda(), labels[keep], eps=eps)


@pytest.mark.parametrize("N", [10, 5000, 70000])
def test_labels_outside(N):
    """A label >= N: NaN in its row and a recorded error, the other rows as they are."""
    x, labels = logits(6, N, F32, 4)
    labels[2], labels[4] = N, 2 ** 40
    check(x.cuda(), labels)
    assert rwo.get_status() == rwo.OK


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("N", [100, 9000, 140000])
def test_large_magnitudes(N, dt):
    """Rows far from 0, one dominant entry, equal entries."""
    x, labels = logits(6, N, F32, 5)
    x[0] += 1e6
    x[1] -= 3e5
    x[2, N // 3] = 1e30
    x[3] = 7.25
    x[4] *= 1e4
    x[5] = -1e30
    check(x.to(dt).cuda(), labels, eps=0.1)


def test_fp16_scaled_gradients():
    """Gradients near fp16's smallest values, and a loss scale that keeps them."""
    x, labels = logits(64, 32000, FP, 6)
    check(x.cuda(), labels, grad_scale=1 / 4096)
    check(x.cuda(), labels, grad_scale=65536 / 64)


def test_leading_dimensions_and_empty():
    x, labels = logits(12, 500, BF, 7)
    want = rwo.cross_entropy_rows_grad(x.cuda(), labels)
    loss, g = rwo.cross_entropy_rows_grad(x.cuda().view(3, 4, 500), labels.view(3, 4))
    assert loss.shape == (3, 4) and g.shape == (3, 4, 500)
    assert torch.equal(loss.view(-1), want[0]) and torch.equal(g.view(12, 500), want[1])
    loss, g = rwo.cross_entropy_rows_grad(x.cuda()[:0], labels[:0])
    assert loss.shape == (0,) and g.shape == (0, 500)


@pytest.mark.parametrize("M,N,dt", [(3000, 64, F32), (2000, 1000, BF), (700, 32768, BF), (400, 50021, F32), (333, 131072, BF), (100, 262145, FP)])
def test_many_rows_agree_with_the_loss_and_repeat(M, N, dt):
    """Many rows of each kernel's range: the loss of cross_entropy_rows, each row as by itself, the same bits again."""
    gen = torch.Generator(device="cuda").manual_seed(9)
    x = (3 * torch.randn(M, N, device="cuda", generator=gen)).to(dt)
    labels = torch.randint(-1, N, (M,), device="cuda", generator=gen)
    lse = torch.empty(M, device="cuda")
    loss, g = rwo.cross_entropy_rows_grad(x, labels, lse_out=lse, grad_scale=0.5)
    again = rwo.cross_entropy_rows_grad(x, labels, grad_scale=0.5)
    assert torch.equal(loss, again[0]) and torch.equal(g, again[1])
    lse2 = torch.empty_like(lse)
    want = rwo.cross_entropy_rows(x, labels, lse_out=lse2)
    assert ((loss - want).abs() <= 2e-5 * want.abs().clamp(min=1)).all() and ((lse - lse2).abs() <= 2e-5 * lse2.abs().clamp(min=1)).all()
    for r in sorted({0, 1, M // 2, M - 1}):
        check(x[r: r + 1], labels[r: r + 1], grad_scale=0.5)
        _, ref, gref, tol = reference(x[r: r + 1], labels[r: r + 1], grad_scale=0.5)
        assert_close(g[r: r + 1], gref, tol + half_step(gref, dt), "grad")
    # softmax minus the label sums to 0 over a row: 1e-5 of the softmax, half a step of what adds up to 2 in all (fp16: at
    # least 2^-25 an element)
    total = g.double().sum(1)
    assert (total.abs() <= 1e-5 + float(torch.finfo(dt).eps) + (N * 2.0 ** -25 if dt is FP else 0)).all()


def test_gradient_against_differences():
    """The formula's gradient, which the kernel is held to above, against central differences of its loss in 64 bits."""
    x, labels = logits(4, 23, F32, 8)
    labels[:] = torch.tensor([3, 0, 22, -1])
    w = torch.tensor([0.5, 2.0, 1.0, 3.0])
    _, _, g, _ = reference(x, labels, w, 1.5, 0.2, 1e-2)
    got = rwo.cross_entropy_rows_grad(x.cuda(), labels, upstream=w.cuda(), grad_scale=1.5, label_smoothing=0.2, z_loss=1e-2)[1].double().cpu()
    h = 1e-5
    for j in range(23):
        e = torch.zeros(23, dtype=torch.float64)
        e[j] = h
        up, down = (reference(x.double() + s * e, labels, w, 1.5, 0.2, 1e-2)[0] for s in (1, -1))
        diff = 1.5 * w.double() * (up - down) / (2 * h)
        assert ((diff - g[:, j]).abs() < 1e-8).all()
        assert ((diff - got[:, j]).abs() < 1e-5 * (1 + 1.5 * w)).all()


def test_streams_and_graphs():
    """Another stream, and a captured call replayed on new logits."""
    x, labels = logits(64, 32768, BF, 10)
    x = x.cuda()
    want = rwo.cross_entropy_rows_grad(x, labels)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = rwo.cross_entropy_rows_grad(x, labels, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    buf = torch.zeros_like(x)
    loss = torch.empty(64, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rwo.cross_entropy_rows_grad(buf, labels, grad=buf, loss=loss)
    for _ in range(2):
        buf.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss, want[0]) and torch.equal(buf, want[1])
