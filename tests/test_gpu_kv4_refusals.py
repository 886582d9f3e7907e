"""Attention over a 4-bit cache: workspaces and hints that the library refuses."""
import pytest
import torch

from speculative_decoding_attention_verify_b200 import sdattn as sd

from .test_gpu_kv4_attention import Call, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 9, 20])
def test_a_workspace_that_is_too_small(rows):
    c = Call([9000], [rows], 14, 2, 128, False)
    need = sd.sd_kv4_attention_workspace_size(c.queries, c.kv)
    assert need > 0
    for n in (0, need - 1):
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        with pytest.raises(sd.SdError) as e:
            sd.sd_kv4_verify_attention(c.queries, c.kv, workspace=ws)
        assert e.value.status == sd.SD_ERR_WORKSPACE


def test_hints_of_no_rows_and_too_many_positions():
    c = Call([30], [2], 4, 1, 64, True)
    for rows, length in ((0, 30), (2, 0), (2, (1 << 30) + 1)):
        with pytest.raises(sd.SdError) as e:
            sd.sd_kv4_verify_attention(sd.Queries(c.queries.q, i32([0, 2]), rows, length), c.kv)
        assert e.value.status == sd.SD_ERR_INVALID_ARG
