"""A chunk of a prompt over a prefix held in 4 bits, with grouped heads and prompts of several lengths: straight from the cache,
and by attention_forward on what kv4_gather reads back, each against 64 bits over the values that the cache holds.

Bound, on the root of the mean square of a sequence's outputs relative to the outputs': a value rounded to the element type is
off by half a step u at most and by u / sqrt(3) in the mean square.  attention_forward sees four such roundings (keys, whose
errors add up to one of the score's own size here, with q and k of about unit variance; weights; values; outputs),
attention_kv4 three at most (weights, weights times scales, outputs), all independent: u sqrt(4 / 3) together.  3 u is asked.
That a bound is able to fail is shown on the oracle: what it gives for mistaken heads, masks and weights is 5 bounds off.
"""
import numpy as np
import pytest
import torch

import row_wise_online_gb300 as rwo
from kv4_reference import Cache, np_of
from test_kv4 import BF, FP, cu_of, dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from row_wise_online_gb300 import _build

    _build.build()
    torch.cuda.set_device(0)


def oracle(k, v, q, sees):
    """q [n, d] over k, v [len, d] in float64; row i sees the first sees[i] keys."""
    z = q @ k.T / np.sqrt(q.shape[1])
    z[np.arange(len(k)) >= np.asarray(sees)[:, None]] = -np.inf
    p = np.exp(z - z.max(1, keepdims=True))
    return p @ v / p.sum(1, keepdims=True)


def off(a, b):
    return np.linalg.norm(a - b) / np.linalg.norm(b)


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("d,heads,group", [(128, 2, 4), (64, 3, 2), (128, 4, 1)])
def test_chunks_over_cached_prefixes(d, heads, group, dt):
    prefix, chunk, hq, page = [333, 40, 0], [70, 129, 61], heads * group, 32
    lens, B = [a + b for a, b in zip(prefix, chunk)], 3
    gen = torch.Generator().manual_seed(d + group)
    T = sum(lens)
    k, v = (torch.randn(T, heads, d, generator=gen).to(dt).cuda() for _ in range(2))
    q = torch.randn(sum(chunk), hq, d, generator=gen).to(dt).cuda()
    pages = [-(-n // page) for n in lens]
    cache, table = rwo.kv4_cache_empty(sum(pages), heads, page, d), np.full((B, max(pages)), -1)
    order = np.random.default_rng(1).permutation(sum(pages))
    for b, n in enumerate(pages):
        table[b, :n], order = order[:n], order[n:]
    where, whole, part = (cache, dev(table), dev(lens)), cu_of(lens), cu_of(chunk)
    rwo.kv4_append(k, v, *where, cu_tokens=dev(whole))
    straight = rwo.attention_kv4(q, *where, cu_tokens=dev(part))
    # read back as [heads][tokens][d]; then a call a sequence, its key/value heads repeated for their query heads
    kk, vv = (torch.empty(heads, T, d, dtype=dt, device="cuda") for _ in range(2))
    rwo.kv4_gather(*where, cu_tokens=dev(whole), k=kk.transpose(0, 1), v=vv.transpose(0, 1))
    back = torch.empty_like(straight)
    for b in range(B):
        rows, held = slice(part[b], part[b + 1]), slice(whole[b], whole[b + 1])
        kb, vb = (x[:, held].repeat_interleave(group, 0) for x in (kk, vv))
        back[rows] = rwo.attention_forward(q[rows].transpose(0, 1).contiguous(), kb, vb, causal=True).transpose(0, 1)
    assert rwo.get_status() == rwo.OK
    bound = 3 * torch.finfo(dt).eps / 2
    c, qf = Cache(cache.cpu().numpy()), np_of(q)
    for b, (n, new) in enumerate(zip(lens, chunk)):
        rows = slice(part[b], part[b + 1])
        sees = n - new + 1 + np.arange(new)
        kv = [c.sequence(table[b], n, h) for h in range(heads)]

        def every_head(head_of, f):
            return np.stack([f(*kv[head_of(h)], qf[rows, h]) for h in range(hq)], 1)

        want = every_head(lambda h: h // group, lambda k, v, x: oracle(k, v, x, sees))
        assert off(np_of(straight)[rows], want) <= bound
        assert off(np_of(back)[rows], want) <= bound
        wrong = [every_head(lambda h: h // group, lambda k, v, x: oracle(k, v, x, [n] * new)),  # no mask
                 every_head(lambda h: h // group, lambda k, v, x: oracle(k, v, x, np.maximum(1, sees - 8))),  # the last keys hidden
                 every_head(lambda h: h // group, lambda k, v, x: oracle(k, v, 0 * x, sees)),  # equal weights
                 every_head(lambda h: heads - 1 - h // group, lambda k, v, x: oracle(k, v, x, sees)),
                 every_head(lambda h: h // group, lambda k, v, x: oracle(k[n // 2:], v[n // 2:], x, np.maximum(1, sees - n // 2))),
                 0 * want]
        assert all(off(x, want) > 5 * bound for x in wrong)
