"""Cache appends without rows, without a GPU: nothing is launched, whatever the empty tensors' addresses."""
import pytest

from speculative_decoding_attention_verify_b200 import sdattn as sd

from .test_kv4_abi import FAKE, _append, _rope, _rows


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("q_out", [None, FAKE])
def test_no_rows_and_no_addresses(q_out, kv4):
    """Empty tensors' data_ptr() is 0."""
    assert _append(rows=_rows(n_rows=0, q=None, k=None, v=None), q_out=q_out, kv4=kv4) == sd.SD_OK
    assert _append(rows=_rows(n_rows=0, h_q=0, q=None, k=None, v=None), q_out=None, kv4=kv4) == sd.SD_OK
    # one row needs them all
    for name in ("q", "k", "v"):
        assert _append(rows=_rows(n_rows=1, **{name: None}), kv4=kv4) == sd.SD_ERR_INVALID_ARG
    # what does not depend on the rows is checked all the same
    assert _append(rows=_rows(n_rows=0, k=None, v=None, max_kv_len=0), kv4=kv4) == sd.SD_ERR_INVALID_ARG
    assert _append(rope=_rope(rotary_dim=3), rows=_rows(n_rows=0, k=None, v=None),
                   kv4=kv4) == sd.SD_ERR_INVALID_ARG
