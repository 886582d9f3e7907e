"""Cache appends: batches without rows, and row starts that do not fit the rows."""
import pytest
import torch

from speculative_decoding_attention_verify_b200 import sdattn as sd

from .test_gpu_kv_append import BF, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("h_q", [0, 4])
def test_empty_tensors(h_q, kv4):
    """No rows at all: nothing is written, and the result has no rows."""
    c = Case([30, 20], [1, 1], h_q, 2, 64, False, BF, kv4=kv4)
    call = sd.sd_kv4_append if kv4 else sd.sd_kv_append
    keep = c.cache.k.clone()
    starts = torch.zeros(3, dtype=torch.int32, device="cuda")
    rows = sd.NewRows(c.dk[:0], c.dv[:0], starts, 31, q=c.dq[:0] if h_q else None)
    q = call(sd.Rope(64), rows, c.cache)
    assert (q is None) if h_q == 0 else q.shape == (0, 4, 64)
    rows = sd.NewRows(c.dk[:0].contiguous(), c.dv[:0].contiguous(), starts, 31)
    assert call(None, rows, c.cache) is None
    assert torch.equal(c.cache.k, keep)
