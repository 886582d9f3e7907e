"""Descriptors of caches and queries refuse tensors whose lengths, tables or types do not fit, before any
pointer is taken (so without a GPU): an append would write where they say."""
import pytest
import torch

from speculative_decoding_attention_verify_b200 import sdattn as sd


def kv(batch=2, kv_len=None, table=None, v=None):
    k = torch.zeros(batch, 4, 16, 64, dtype=torch.bfloat16)
    kv_len = torch.zeros(2, dtype=torch.int32) if kv_len is None else kv_len
    return sd.KVCache(k, k.clone() if v is None else v, kv_len, table)


def test_more_lengths_than_sequences():
    with pytest.raises(ValueError, match="more sequences"):
        kv(batch=1)
    with pytest.raises(ValueError, match="more sequences"):
        kv(batch=9, table=torch.zeros(1, 3, dtype=torch.int32))


def test_lengths_and_pages_of_other_types_and_shapes():
    with pytest.raises(ValueError, match="kv_len must be"):
        kv(kv_len=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="kv_len must be"):
        kv(kv_len=torch.zeros(2, 1, dtype=torch.int32))
    with pytest.raises(ValueError, match="block_table must be"):
        kv(table=torch.zeros(2, 3, dtype=torch.int64))
    with pytest.raises(ValueError, match="block_table must be"):
        kv(table=torch.zeros(6, dtype=torch.int32))


def test_tensors_of_several_devices():
    meta = lambda *s, t=torch.int32: torch.zeros(*s, dtype=t, device="meta")  # noqa: E731
    with pytest.raises(ValueError, match="one device"):
        kv(kv_len=meta(2))
    with pytest.raises(ValueError, match="one device"):
        kv(table=meta(2, 3))
    with pytest.raises(ValueError, match="one device"):
        kv(v=meta(2, 4, 16, 64, t=torch.bfloat16))


def test_what_fits_goes_on_to_the_next_check():
    """(CPU tensors are refused last)"""
    for kw in (dict(), dict(batch=3), dict(table=torch.zeros(5, 3, dtype=torch.int32))):
        with pytest.raises(ValueError, match="on the GPU"):
            kv(**kw)


def test_row_starts_of_queries():
    """(an int64 vector would be read as twice as many sequences' starts)"""
    q = torch.zeros(4, 8, 64, dtype=torch.bfloat16)
    for bad in (torch.zeros(3, dtype=torch.int64), torch.zeros(3, 1, dtype=torch.int32),
                torch.zeros(3, dtype=torch.int32, device="meta")):
        with pytest.raises(ValueError, match="q_start must be"):
            sd.Queries(q, bad, 2, 16)
    with pytest.raises(ValueError, match="on the GPU"):
        sd.Queries(q, torch.zeros(3, dtype=torch.int32), 2, 16)
