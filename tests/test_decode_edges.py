"""Calls of the decoding step at the ends of what they take."""
import numpy as np
import pytest
import torch

import row_wise_online_gb300 as rwo
from test_kv4 import BF, FP, check_attention, dev, pool

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from row_wise_online_gb300 import _build

    _build.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("d,group", [(128, 1), (64, 12)])
@pytest.mark.parametrize("q_sd,scale", [(1e30, 1e-30), (1e37, 1e-37), (0.0, 1e-30), (0.0, 3e38), (1e-37, 1e37), (3e-39, 2e38), (1.0, 1e-30)])
def test_scales_and_queries_far_from_one(q_sd, scale, d, group):
    """scale q is of ordinary size, or of none: the scores are finite, whatever the two are."""
    lens = [900, 33, 2000]
    c, table = pool(lens, 2, 16, d, seed=d)
    check_attention(c, table, lens, [1, 3, 2], 2 * group, BF, seed=3, q_sd=q_sd, scale=scale)


@pytest.mark.parametrize("runs", [False, True])
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("d,group", [(128, 4), (64, 2)])
def test_tokens_that_are_not_numbers(d, group, dt, runs):
    """A last token of NaN and infinities: the cache stays finite, the bytes of every other group and the rows of every
    other token what they are without it."""
    n, heads = 40, 2
    gen = torch.Generator().manual_seed(d)
    k, v = (torch.randn(n, heads, d, generator=gen).to(dt).cuda() for _ in range(2))
    q = torch.randn(4, heads * group, d, generator=gen).to(dt).cuda()
    table, lens = dev([[2, 0, 1]]), dev([n])
    held, out = [], []
    for bad in (False, True):
        cache = rwo.kv4_cache_empty(3, heads, 16, d)
        rwo.kv4_append(k[:n - 1], v[:n - 1], cache, table, lens - 1, cu_tokens=dev([0, n - 1]))
        kk, vv = k.clone(), v.clone()
        if bad:
            kk[n - 1, 0, :] = float("nan")
            vv[n - 1, 0, :32] = float("nan")
            vv[n - 1, 0, 32:64] = float("inf")
            vv[n - 1, 1, 3] = float("nan")
            vv[n - 1, 1, 34] = -float("inf")
        if runs:  # many tokens a sequence: the last ones are written again
            rwo.kv4_append(kk[n - 9:], vv[n - 9:], cache, table, lens, cu_tokens=dev([0, 9]))
        else:
            rwo.kv4_append(kk[n - 1:], vv[n - 1:], cache, table, lens)
        held.append([t[:n - 1] for t in rwo.kv4_gather(cache, table, lens, cu_tokens=dev([0, n]), num_tokens=n, dtype=dt)])
        assert np.isfinite(cache.cpu().numpy().view(np.float16)[..., 8 * d:]).all()
        out.append(rwo.attention_kv4(q, cache, table, lens, cu_tokens=dev([0, 4])))
        assert rwo.get_status() == rwo.OK
    assert all(torch.equal(a, b) for a, b in zip(*held))
    assert torch.equal(out[0][:3], out[1][:3])


@pytest.mark.parametrize("repetition", [1.3, 0.7, 1e-41, 3e38])
def test_repetition_divides(repetition):
    """A seen logit above zero is divided, one below multiplied: the fp32 quotient and product, to the last bit."""
    M, N = 3, 4097
    gen = torch.Generator().manual_seed(1)
    x = 3 * torch.randn(M, N, generator=gen)
    x[0, :9] = torch.tensor([1e-45, -1e-45, 1e-39, -1e-39, 0.0, 3e38, -3e38, 1e-3, 7.0])
    rep = torch.full((M,), repetition)
    tokens = torch.arange(N, dtype=torch.int32).repeat(M, 1)
    y = rwo.logits_process_rows(x.cuda(), out="logits", tokens=tokens.cuda(), token_lens=dev([N] * M), repetition=rep.cuda())
    assert rwo.get_status() == rwo.OK
    r = rep.numpy()[:, None]
    with np.errstate(over="ignore"):
        want = np.where(x.numpy() > 0, x.numpy() / r, x.numpy() * r)
    assert np.array_equal(y.cpu().numpy(), want)


def test_offsets_that_descend_are_not_worked_on():
    """Offsets 0, T, 0, T, ...: half of the sequences claim every row.  Reported, and no row is written."""
    T, B, heads, d = 20000, 2000, 4, 64
    data = rwo.kv4_cache_empty(1, heads, 65536, d)
    q = torch.zeros(T, 2 * heads, d, dtype=BF, device="cuda")
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1::2] = T
    lens = torch.full((B,), 65536, dtype=torch.int32, device="cuda")
    o, lse = torch.full_like(q, 3.0), torch.full((T, 2 * heads), 3.0, device="cuda")
    ws = rwo.attention_kv4_workspace(B, T, 2 * heads, heads, d)
    ws.fill_(255)
    rwo.attention_kv4(q, data, torch.zeros(B, 1, dtype=torch.int32, device="cuda"), lens, cu_tokens=cu, o=o, lse_out=lse, workspace=ws)
    assert rwo.get_status() == rwo.ERR_INVALID_ARG
    assert (o == 3).all() and (lse == 3).all()
