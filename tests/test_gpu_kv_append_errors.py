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


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("starts,good", [([-2, 4, 8], 1), ([0, 4, 12], 0), ([0, 8, 12], 0),
                                         ([-4, 0, 8], 1), ([8, 9, 10], None),
                                         ([0, 8, 4], 0), ([-2**31, 2**31 - 1, 8], None)])
def test_row_starts_outside_the_rows(starts, good, wide, kv4):
    """8 rows.  A sequence that begins before them, ends behind them or ends before it begins is
    reported and skipped, whether or not a row of the tensor falls into it; the other one is not
    (where starts decrease, its rows may be skipped too)."""
    c = Case([30, 20], [8, 8], 4, 2, 64, False, BF, slack=0 if wide else 1, kv4=kv4)
    c.kv_len.copy_(torch.tensor([38, 28], dtype=torch.int32))
    call = sd.sd_kv4_append if kv4 else sd.sd_kv_append
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
    q_out = torch.full((8, 4, 64), 9.0, dtype=BF, device="cuda")
    call(sd.Rope(64), sd.NewRows(c.dk[:8], c.dv[:8], q_start, 38, q=c.dq[:8]), c.cache,
         q_out=q_out, dev_err=flag)
    torch.cuda.synchronize()
    assert flag.item() == sd.SD_DEVERR_SHAPE
    k = (c.cache.k_param if kv4 else c.cache.k).cpu()
    touched = (k != 7).any(-1).any(1)  # [sequence][position]
    want = torch.zeros_like(touched)
    rows = torch.zeros(8, dtype=torch.bool)
    if good is not None:
        n, end = starts[good + 1] - starts[good], (38, 28)[good]
        want[good, end - n:end] = True
        rows[starts[good]:starts[good + 1]] = True
    turned = (q_out.cpu() != 9).any(-1).any(-1)
    if starts == sorted(starts):
        assert torch.equal(touched, want) and torch.equal(turned, rows)
    else:
        assert not (touched & ~want).any() and not (turned & ~rows).any()


@pytest.mark.parametrize("kv4", [False, True])
def test_a_bad_start_far_down_a_large_batch(kv4):
    """More sequences than a block has threads; the last one lies behind the rows."""
    n = 700
    c = Case([0] * n, [1] * n, 2, 1, 64, False, BF, kv4=kv4)
    call = sd.sd_kv4_append if kv4 else sd.sd_kv_append
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = sd.NewRows(c.dk[:n - 1], c.dv[:n - 1], c.q_start, 1)
    call(None, rows, c.cache, dev_err=flag)
    torch.cuda.synchronize()
    assert flag.item() == sd.SD_DEVERR_SHAPE
    k = (c.cache.k_param if kv4 else c.cache.k).cpu()
    assert (k[:n - 1, :, 0] != 7).any(-1).all() and (k[n - 1] == 7).all()
    flag.zero_()
    call(None, c.new_rows(q=False), c.cache, dev_err=flag)
    assert flag.item() == 0
