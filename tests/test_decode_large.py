"""The decoding-step calls where byte and element offsets pass 32 bits: the same values as in a small place."""
import pytest
import torch

import row_wise_online_gb300 as rwo

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from row_wise_online_gb300 import _build

    _build.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("news", [None, [40, 9, 200]])
def test_pages_behind_4_gib(news):
    """A pool of 5 GiB of which the last pages are used, against the same pages in a small pool; rows at a token stride of
    2^30 + 64 elements, so that the third begins behind 4 GiB."""
    heads, group, d, page = 2, 2, 128, 64
    lens = [130, 64, 257]
    need = [-(-n // page) for n in lens]
    pages = 5 * 2 ** 30 // (heads * page // 16 * 20 * d)
    small, large = rwo.kv4_cache_empty(sum(need), heads, page, d), rwo.kv4_cache_empty(pages, heads, page, d)
    table, at = torch.zeros(3, max(need), dtype=torch.int32, device="cuda"), 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n)
        at += n
    far = table + (pages - at)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    fill = torch.tensor([0, 130, 194, 451], dtype=torch.int32, device="cuda")
    k, v = (torch.randn(451, heads, d, generator=gen, device="cuda").to(BF) for _ in range(2))
    for cache, tab in ((small, table), (large, far)):
        rwo.kv4_append(k, v, cache, tab, ln, cu_tokens=fill)
    cu = None if news is None else torch.tensor([0, 40, 49, 249], dtype=torch.int32, device="cuda")
    T = 3 if news is None else 249
    q = torch.randn(T, heads * group, d, generator=gen, device="cuda").to(BF)
    wide = q
    if news is None:  # rows far apart
        buf = torch.empty(2 * (2 ** 30 + 64) + heads * group * d, dtype=BF, device="cuda")
        wide = buf.as_strided((3, heads * group, d), (2 ** 30 + 64, d, 1))
        wide.copy_(q)
    a, b = (rwo.attention_kv4(x, cache, tab, ln, cu_tokens=cu) for x, cache, tab in ((q, small, table), (wide, large, far)))
    assert rwo.get_status() == rwo.OK
    assert torch.equal(a, b)
    ka, va = rwo.kv4_gather(small, table, ln, cu_tokens=cu, num_tokens=T)
    kb, vb = rwo.kv4_gather(large, far, ln, cu_tokens=cu, num_tokens=T)
    assert torch.equal(ka, kb) and torch.equal(va, vb) and ka.any()
    assert torch.equal(large[pages - at:], small) and not large[:pages - at].any()


def test_keys_far_apart():
    """Keys and values at a token stride behind 4 GiB, by rows and in runs."""
    heads, d, stride = 1, 64, 2 ** 29 + 64
    gen = torch.Generator(device="cuda").manual_seed(2)
    for T, cu in ((3, None), (6, [0, 6])):
        n = T if cu is None else 1
        k = torch.randn(T, heads, d, generator=gen, device="cuda").to(BF)
        buf = torch.empty((T - 1) * stride + d, dtype=BF, device="cuda")
        far = buf.as_strided((T, heads, d), (stride, d, 1))
        far.copy_(k)
        table = torch.arange(n, dtype=torch.int32, device="cuda")[:, None]
        ln = torch.full((n,), 7, dtype=torch.int32, device="cuda")
        c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
        near, there = rwo.kv4_cache_empty(n, heads, 16, d), rwo.kv4_cache_empty(n, heads, 16, d)
        rwo.kv4_append(k, k, near, table, ln, cu_tokens=c)
        rwo.kv4_append(far, far, there, table, ln, cu_tokens=c)
        assert torch.equal(near, there) and near.any()
        out = torch.empty_like(buf).as_strided((T, heads, d), (stride, d, 1))
        rwo.kv4_gather(near, table, ln, cu_tokens=c, k=out, v=torch.empty_like(k))
        assert torch.equal(out, rwo.kv4_gather(near, table, ln, cu_tokens=c, num_tokens=T)[0])
        assert rwo.get_status() == rwo.OK


def test_logits_rows_far_apart():
    N, pitch = 5000, 2 ** 31 + 8
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(2, N, generator=gen, device="cuda").to(BF)
    buf = torch.empty(pitch + N, dtype=BF, device="cuda")
    far = buf.as_strided((2, N), (pitch, 1))
    far.copy_(x)
    opts = dict(tokens=torch.randint(0, N, (2, 50), generator=gen, device="cuda", dtype=torch.int32),
                token_lens=torch.tensor([50, 20], dtype=torch.int32, device="cuda"), frequency=torch.tensor([0.3, 0.1], device="cuda"))
    want = rwo.logits_process_rows(x, **opts)
    assert torch.equal(rwo.logits_process_rows(far, **opts), want)
    rwo.logits_process_rows(far, y=far, **opts)
    assert torch.equal(far, want)
    assert rwo.get_status() == rwo.OK
