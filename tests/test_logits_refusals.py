"""logits_process_rows without a GPU: a pointer that is not aligned to its elements is refused before anything is enqueued."""
import pytest

import row_wise_online_gb300 as rwo
from row_wise_online_gb300 import _build, decode

X = 0x10000  # never dereferenced: every call below fails validation first


@pytest.mark.parametrize("name", ["lse_out", "tokens", "prompt_lens", "token_lens", "repetition", "frequency", "presence",
                                  "bias_ids", "bias_values", "mask", "scale"])
def test_pointers_off_their_elements(name):
    _build.build()
    given = dict(x=X, y=X, tokens=X, token_width=5, token_lens=X, bias_ids=X, bias_values=X, bias_count=2)
    for off in (1, 2, 3):
        a = decode._Logits(**{**given, name: X + off})
        assert rwo.capi().logits_process_rows(a, 4, 100, 0, 1, None) == rwo.ERR_MISALIGNED
