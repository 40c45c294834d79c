"""The decoding-step calls without a GPU: every argument that the host can refuse is refused before anything is enqueued."""
import ctypes

import pytest
import torch

import row_wise_online_gb300 as rwo
from row_wise_online_gb300 import _build, decode

X = 0x10000  # never dereferenced: every call below fails validation first
BAD, ODD, NO, OK = rwo.ERR_INVALID_ARG, rwo.ERR_MISALIGNED, rwo.ERR_UNSUPPORTED, rwo.OK


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return rwo.capi()


def cache(**kw):
    a = dict(data=X, page_table=X, seq_lens=X, cu_tokens=None, num_pages=8, page_size=16, heads=2, head_dim=128, batch=3,
             table_width=4, tokens=3)
    a.update(kw)
    return decode._Cache(**a)


def rows(p=X, token=256, head=128):
    return decode._Rows(p, token, head)


CACHE_FAULTS = [
    (dict(head_dim=96), NO), (dict(head_dim=0), BAD), (dict(page_size=24), NO), (dict(page_size=0), BAD), (dict(heads=0), BAD),
    (dict(batch=-1), BAD), (dict(tokens=-1), BAD), (dict(num_pages=-1), BAD), (dict(table_width=-1), BAD),
    (dict(tokens=4), BAD),  # no cu_tokens: one row a sequence
    (dict(num_pages=0), BAD), (dict(table_width=0), BAD), (dict(data=None), BAD), (dict(page_table=None), BAD),
    (dict(seq_lens=None), BAD), (dict(data=X + 8), ODD), (dict(page_table=X + 2), ODD), (dict(seq_lens=X + 1), ODD),
    (dict(cu_tokens=X + 2), ODD), (dict(table_width=2 ** 28), NO), (dict(page_size=2 ** 40), NO), (dict(num_pages=2 ** 40), NO),
    (dict(heads=2 ** 17), NO), (dict(batch=2 ** 25, tokens=2 ** 25), NO), (dict(cu_tokens=X, tokens=2 ** 31), NO),
]


@pytest.mark.parametrize("kw,want", CACHE_FAULTS)
def test_cache_faults(lib, kw, want):
    c = cache(**kw)
    assert lib.kv4_append(c, rows(), rows(), None, None, 0, None, 0, 0, 0, 1, None) == want
    assert lib.kv4_gather(c, rows(), rows(), 1, None) == want
    assert lib.attention_kv4(c, rows(), X, None, 4 * max(1, c.heads) if c.heads < 1000 else c.heads, 0.0, 1, X, 2 ** 40, None) == want


def test_no_tokens_is_a_no_op(lib):
    for kw in (dict(batch=0, tokens=0), dict(cu_tokens=X, tokens=0), dict(batch=0, tokens=5, cu_tokens=X)):
        c = cache(data=None, page_table=None, seq_lens=None, num_pages=0, **kw)
        assert lib.kv4_append(c, None, None, None, None, 0, None, 0, 0, 0, 1, None) == OK
        assert lib.kv4_gather(c, None, None, 2, None) == OK
        assert lib.attention_kv4(c, None, None, None, 4, 0.0, 2, None, 0, None) == OK
    assert lib.attention_kv4_workspace(0, 0, 4, 2, 128) == 0


def test_append_faults(lib):
    def call(c=None, k=rows(), v=rows(), q=None, qo=None, heads=0, cs=None, pos=0, rot=0, flags=0, dt=1):
        return lib.kv4_append(c or cache(), k, v, q, qo, heads, cs, pos, rot, flags, dt, None)

    assert lib.kv4_append(None, rows(), rows(), None, None, 0, None, 0, 0, 0, 1, None) == BAD
    assert call(dt=0) == NO and call(dt=5) == BAD
    assert call(k=None) == BAD and call(v=rows(None)) == BAD
    assert call(k=rows(X + 8)) == ODD and call(v=rows(X, 260)) == ODD and call(v=rows(X, 256, 132)) == ODD
    assert call(q=rows()) == BAD and call(qo=rows(), heads=4) == BAD  # one without the other
    assert call(q=rows(), qo=rows(), heads=0) == BAD and call(q=rows(X + 2), qo=rows(), heads=4) == ODD
    assert call(flags=2) == BAD
    assert call(cs=X, pos=8, rot=0) == BAD and call(cs=X, pos=8, rot=136) == BAD and call(cs=X, pos=0, rot=64) == BAD
    assert call(cs=X, pos=8, rot=60) == NO and call(cs=X + 4, pos=8, rot=64) == ODD
    assert call(k=rows(X, 2 ** 62)) == BAD


def test_gather_and_attention_faults(lib):
    assert lib.kv4_gather(cache(), rows(), rows(), 0, None) == NO
    assert lib.kv4_gather(cache(), rows(X + 4), rows(), 1, None) == ODD

    def att(q=rows(), o=X, lse=None, heads=4, scale=0.0, dt=1, ws=X):
        return lib.attention_kv4(cache(), q, o, lse, heads, scale, dt, ws, 2 ** 40, None)

    assert att(heads=3) == BAD and att(heads=0) == BAD  # not a multiple of the key/value heads
    assert att(scale=-1.0) == BAD and att(scale=float("nan")) == BAD and att(scale=float("inf")) == BAD
    assert att(dt=0) == NO and att(dt=9) == BAD
    assert att(q=None) == BAD and att(o=None) == BAD and att(ws=None) == BAD
    assert att(o=X + 8) == ODD and att(ws=X + 16) == ODD and att(lse=X + 2) == ODD and att(q=rows(X, 100)) == ODD
    assert lib.attention_kv4_workspace(1, 1, 3, 2, 128) == -1 and lib.attention_kv4_workspace(1, 1, 4, 2, 96) == -1


def test_logits_faults(lib):
    def call(M=4, N=100, dt=0, out=1, **kw):
        a = decode._Logits(**{**dict(x=X, y=X), **kw})
        return lib.logits_process_rows(a, M, N, dt, out, None)

    assert lib.logits_process_rows(None, 4, 4, 0, 1, None) == BAD
    assert call(N=0) == BAD and call(M=-1) == BAD and call(dt=7) == BAD and call(out=3) == BAD and call(out=-1) == BAD
    assert call(x=None) == BAD and call(y=None) == BAD
    assert call(ldx=99) == BAD and call(ldy=99) == BAD and call(mask=X, ld_mask=3) == BAD
    assert call(tokens=X, token_width=5) == BAD  # no lengths
    assert call(tokens=X, token_width=-1, token_lens=X) == BAD and call(tokens=X, token_width=2 ** 20, token_lens=X) == NO
    assert call(bias_count=3) == BAD and call(bias_count=1025, bias_ids=X, bias_values=X) == NO and call(bias_count=-1) == BAD
    assert call(x=X + 2) == ODD and call(dt=1, y=X + 1) == ODD
    assert call(N=2 ** 31) == NO and call(M=2 ** 27) == NO and call(M=2 ** 40, N=2 ** 30) in (BAD, NO)
    assert call(M=0, x=None, y=None) == OK


def test_binding_refuses_on_the_host():
    c = torch.zeros(2, 1, 1, 20 * 64, dtype=torch.uint8)
    i = torch.zeros(1, 1, dtype=torch.int32)
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    for call in (lambda: rwo.attention_kv4(q, c, i, i[0]), lambda: rwo.kv4_append(q, q, c, i, i[0]), lambda: rwo.kv4_gather(c, i, i[0])):
        with pytest.raises(ValueError):
            call()  # not CUDA tensors
    with pytest.raises(ValueError):
        rwo.logits_process_rows(torch.zeros(2, 4))
    with pytest.raises(ValueError):
        rwo.logits_process_rows(torch.zeros(2, 4), out="argmax")
    for args in ((4, 2, 24, 64), (4, 2, 0, 64), (4, 2, 16, 96)):
        with pytest.raises(ValueError):
            rwo.kv4_cache_empty(*args, device="cpu")
    assert rwo.kv4_cache_empty(4, 2, 48, 64, device="cpu").shape == (4, 2, 3, 1280)


def test_structures_match_the_header(lib):
    assert ctypes.sizeof(decode._Cache) == 11 * 8 and ctypes.sizeof(decode._Rows) == 24 and ctypes.sizeof(decode._Logits) == 18 * 8
