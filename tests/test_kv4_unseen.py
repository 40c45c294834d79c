"""What a row of attention_kv4 must not see has no part in it, to the last bit: slots of a page that hold no token, and the
keys, values and queries of later tokens.  The same arithmetic on the same inputs: results are compared for equality."""
import numpy as np
import pytest
import torch

import row_wise_online_gb300 as rwo
from kv4_reference import Cache
from test_kv4 import BF, FP, cu_of, dev, pool

pytestmark = pytest.mark.gpu
SHAPES = [(128, 2, 1), (128, 2, 8), (128, 1, 16), (64, 2, 4), (64, 1, 12)]  # d, kv heads, query heads of each


@pytest.fixture(scope="module", autouse=True)
def _built():
    from row_wise_online_gb300 import _build

    _build.build()
    torch.cuda.set_device(0)


def bytes_of(c: Cache, codes_of_v_alone: bool = False) -> np.ndarray:
    """[16][20 d]: which bytes of a block belong to a token."""
    out = np.zeros((16, 20 * c.d), bool)
    for r in range(16):
        out[r, c.v_nibble[r] // 2] = True
        if not codes_of_v_alone:
            out[r, c.k_nibble[r] // 2] = True
            for hf in (c.k_half[r], c.v_half[r]):
                for at in (2 * hf, 2 * (hf + 16 * c.G)):
                    out[r, at] = out[r, at + 1] = True
    return out


def places(c: Cache, table, spans, which) -> np.ndarray:
    """Bytes of the cache [pages][1][blocks][20 d] that tokens [lo, hi) of each sequence have."""
    out = np.zeros((c.data.shape[0], 1) + c.data.shape[2:], bool)
    for row, (lo, hi) in zip(table, spans):
        for pos in range(lo, hi):
            out[row[pos // c.page], 0, pos % c.page // 16] |= which[pos % 16]
    return out


def results(data, table, lens, news, q):
    lse = torch.empty(q.shape[:2], device="cuda")
    o = rwo.attention_kv4(q, torch.from_numpy(data).cuda(), dev(table), dev(lens), cu_tokens=dev(cu_of(news)), lse_out=lse)
    assert rwo.get_status() == rwo.OK
    return o, lse


@pytest.mark.parametrize("d,heads,group", SHAPES)
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("drafts", [1, 3])
def test_slots_that_hold_no_token(drafts, dt, d, heads, group):
    rng = np.random.default_rng(d + group)
    lens = list(range(1, 101)) + [int(n) for n in rng.integers(100, 900, 60)]
    news = [min(n, drafts) for n in lens]
    c, table = pool(lens, heads, 48, d, seed=d + group)
    used = places(c, table, [(0, n) for n in lens], bytes_of(c))
    q = torch.randn(sum(news), heads * group, d, generator=torch.Generator().manual_seed(group)).to(dt).cuda()
    want = results(c.data, table, lens, news, q)  # NaN scales and zeros there
    noise = rng.integers(0, 256, c.data.shape, dtype=np.uint8)
    large = noise.copy()
    large.view(np.float16)[..., 8 * d:] = 65504.0
    for other in (noise, large, np.zeros_like(noise)):
        got = results(np.where(used, c.data, other), table, lens, news, q)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("d,heads,group", SHAPES)
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("change", ["codes of values", "keys and values", "queries"])
def test_later_tokens(change, dt, d, heads, group):
    lens = [9, 33, 64, 100, 260, 700, 131, 1500, 40, 18]
    news = [9, 5, 4, 8, 8, 3, 4, 2, 40, 17]
    keep = [4, 1, 3, 1, 7, 1, 2, 1, 21, 9]  # of the new tokens, those whose rows are compared
    c, table = pool(lens, heads, 32, d, seed=d + group)
    gen = torch.Generator().manual_seed(group)
    q = torch.randn(sum(news), heads * group, d, generator=gen).to(dt).cuda()
    want = results(c.data, table, lens, news, q)
    cu = cu_of(news)
    rows = torch.cat([torch.arange(cu[b], cu[b] + k) for b, k in enumerate(keep)]).cuda()
    later = places(c, table, [(n - new + k, n) for n, new, k in zip(lens, news, keep)], bytes_of(c, change == "codes of values"))
    for seed, factor in ((1, 1.0), (2, 300.0), (3, 0.01)):
        data, other = c.data, np.random.default_rng(seed).integers(0, 256, c.data.shape, dtype=np.uint8)
        half = other.view(np.float16)
        half[..., 8 * d:] = np.random.default_rng(seed).uniform(0.1, 1.0, half[..., 8 * d:].shape) * factor
        if change == "queries":
            hidden = torch.ones(len(q), dtype=torch.bool)
            hidden[rows.cpu()] = False
            q2 = q.clone()
            q2[hidden.cuda()] *= 30.0 * min(factor, 3.0)
        else:
            data, q2 = np.where(later, other, c.data), q
        got = results(data, table, lens, news, q2)
        assert all(torch.equal(a[rows], b[rows]) for a, b in zip(got, want))
