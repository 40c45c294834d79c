"""The training-step calls together, as a program uses them: a small language model of one residual block around two products,
its loss and every gradient against the same model in 64 bits with torch's own differentiation; captured and replayed; two
steps at once on two streams.

Tolerances: fp32 throughout but for the products, which torch does in fp32 (their rounding grows with the square root of their
length).  The gradients of one step are within 1e-4 of their largest entry, the loss within 1e-5 of itself.
"""
import math

import pytest
import torch

import row_wise_online_gb300 as rwo
from train_util import BF, F32

pytestmark = pytest.mark.gpu
T, V, D = 300, 1003, 96


@pytest.fixture(scope="module", autouse=True)
def _built():
    from row_wise_online_gb300 import _build

    _build.build()
    torch.cuda.set_device(0)


def model(seed=0, dt=F32):
    gen = torch.Generator().manual_seed(seed)
    p = {"table": 0.3 * torch.randn(V, D, generator=gen), "w1": 1 + 0.1 * torch.randn(D, generator=gen), "w2": 1 + 0.1 * torch.randn(D, generator=gen),
         "a": torch.randn(D, D, generator=gen) / math.sqrt(D), "b": torch.randn(D, V, generator=gen) / math.sqrt(D)}
    tokens, labels = torch.randint(0, V, (2, T), generator=gen)
    tokens[5] = -1
    labels[::7] = -100
    return {k: v.to(dt).cuda() for k, v in p.items()}, tokens.cuda(), labels.cuda()


SCALE, EPS, Z = 0.1, 1e-5, 1e-3


def step(p, tokens, labels, max_norm):
    """One step's loss and clipped gradients through the library; products by torch."""
    x = rwo.embedding_rows(p["table"], tokens, scale=8.0)
    r1, r2 = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    y1, _ = rwo.rms_norm_rows(x, p["w1"], rstd_out=r1, eps=EPS)
    m = y1 @ p["a"]
    y2, h = rwo.rms_norm_rows(m, p["w2"], residual=x, rstd_out=r2, eps=EPS)
    logits = y2 @ p["b"]
    losses, dl = rwo.cross_entropy_rows_grad(logits, labels, grad=logits, grad_scale=1 / T, label_smoothing=SCALE, z_loss=Z)
    g = {"b": y2.t() @ dl}
    dh, g["w2"] = rwo.rms_norm_rows_backward(dl @ p["b"].t(), h, r2, p["w2"])
    g["a"] = y1.t() @ dh
    dx, g["w1"] = rwo.rms_norm_rows_backward(dh @ p["a"].t(), x, r1, p["w1"], sum_grad=dh)
    g["table"] = rwo.embedding_rows_backward(dx, tokens, V, scale=8.0, dtype=p["table"].dtype)
    names = sorted(g)
    norm = rwo.clip_grad_norm([g[k].contiguous() for k in names], max_norm, out=(out := [torch.empty_like(g[k]) for k in names]))
    return losses, norm, dict(zip(names, out))


def reference(p, tokens, labels, max_norm):
    q = {k: v.detach().double().cpu().requires_grad_() for k, v in p.items()}
    tokens, labels = tokens.cpu(), labels.cpu()

    def norm(x, w):
        return x / torch.sqrt(x.pow(2).mean(1, keepdim=True) + EPS) * w

    x = torch.where((tokens >= 0)[:, None], q["table"][tokens.clamp(min=0)] * 8.0, 0.0)
    h = norm(x, q["w1"]) @ q["a"] + x
    logits = norm(h, q["w2"]) @ q["b"]
    lse = torch.logsumexp(logits, 1)
    logp = logits - lse[:, None]
    losses = -(1 - SCALE) * logp.gather(1, labels.clamp(min=0)[:, None])[:, 0] - SCALE * logp.mean(1) + Z * lse ** 2
    losses = torch.where(labels >= 0, losses, 0.0)
    (losses.sum() / T).backward()
    total = math.sqrt(sum(float(v.grad.pow(2).sum()) for v in q.values()))
    return losses.detach(), total, {k: v.grad * min(1.0, max_norm / total) for k, v in q.items()}


@pytest.mark.parametrize("max_norm", [0.05, 1e6])
def test_step_against_64_bits(max_norm):
    # products in fp32, not in the tensor cores' shorter formats
    held = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        p, tokens, labels = model()
        losses, norm, g = step(p, tokens, labels, max_norm)
    finally:
        torch.backends.cuda.matmul.allow_tf32 = held
    assert rwo.get_status() == rwo.OK
    want, total, ref = reference(p, tokens, labels, max_norm)
    assert ((losses.double().cpu() - want).abs() <= 1e-5 * want.abs().clamp(min=1)).all()
    assert abs(float(norm) - total) <= 1e-4 * total
    for k in g:
        assert (g[k].double().cpu() - ref[k]).abs().max() <= 1e-4 * ref[k].abs().max(), k


def test_step_in_16_bits_runs_and_points_the_same_way():
    p, tokens, labels = model(1, BF)
    losses, norm, g = step(p, tokens, labels, 1e6)
    assert rwo.get_status() == rwo.OK
    want, total, ref = reference(p, tokens, labels, 1e6)
    assert ((losses.double().cpu() - want).abs() <= 0.05 * want.abs().clamp(min=1)).all()  # logits in bf16: 2^-8 of up to 10 each
    for k in g:
        a, b = g[k].double().cpu().flatten(), ref[k].flatten()
        assert (a @ b) / (a.norm() * b.norm()) > 0.99, k


def test_step_captured_and_replayed():
    """The step in a graph, which allocates its workspaces from the graph's own pool, on new tokens and on the old ones."""
    p, tokens, labels = model(2)
    other = model(3)[1:]
    want = [step(p, *b, 0.1) for b in ((tokens, labels), other)]
    buf = tokens.clone(), labels.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        losses, norm, g = step(p, *buf, 0.1)
    second = torch.cuda.CUDAGraph()
    with torch.cuda.graph(second):
        losses2, norm2, g2 = step(p, *buf, 0.1)
    for k in (1, 0, 1):
        for b, t in zip(buf, ((tokens, labels), other)[k]):
            b.copy_(t)
        torch.cuda.synchronize()
        # two captured steps at once
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            second.replay()
        graph.replay()
        torch.cuda.synchronize()
        for got in ((losses, norm, g), (losses2, norm2, g2)):
            assert torch.equal(got[0], want[k][0]) and torch.equal(got[1], want[k][1])
            assert all(torch.equal(got[2][n], want[k][2][n]) for n in g)
    assert rwo.get_status() == rwo.OK


def test_two_steps_at_once():
    """Eager steps on two streams, many times over: each call has a workspace of its own."""
    batches = [model(4), model(5)]
    want = [step(*b, 0.1) for b in batches]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in batches]
    got = [[], []]
    for _ in range(8):
        for k, (s, b) in enumerate(zip(streams, batches)):
            with torch.cuda.stream(s):
                got[k].append(step(*b, 0.1))
    torch.cuda.synchronize()
    for k in range(2):
        for losses, norm, g in got[k]:
            assert torch.equal(losses, want[k][0]) and torch.equal(norm, want[k][1])
            assert all(torch.equal(g[n], want[k][2][n]) for n in g)


def test_streams_given_and_current():
    """stream= as an object and as a pointer; what is allocated for the call belongs to it."""
    p, tokens, labels = model(6)
    s = torch.cuda.Stream()
    want = rwo.embedding_rows_backward(p["table"][:T], tokens, V)
    for given in (s, s.cuda_stream):
        s.wait_stream(torch.cuda.current_stream())
        a = rwo.embedding_rows(p["table"], tokens, stream=given)
        b = rwo.embedding_rows_backward(p["table"][:T], tokens, V, stream=given)
        c = rwo.grad_norm([p["a"], p["b"]], stream=given)
        y, _ = rwo.rms_norm_rows(p["a"], p["w1"], stream=given)
        s.synchronize()
        assert torch.equal(a, rwo.embedding_rows(p["table"], tokens)) and torch.equal(b, want)
        assert torch.equal(c, rwo.grad_norm([p["a"], p["b"]])) and torch.equal(y, rwo.rms_norm_rows(p["a"], p["w1"])[0])
