"""Calls of the decoding step at the ends of what they take."""
import numpy as np
import pytest
import torch

import row_wise_online_gb300 as rwo
from test_kv4 import BF, check_attention, pool

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
