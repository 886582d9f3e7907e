"""The longest context of attention over a 4-bit cache, without a GPU: positions are 32-bit, and a tile's
end behind the last one has to be one too."""
import ctypes

import pytest

from speculative_decoding_attention_verify_b200 import sdattn as sd

from .test_kv4_abi import _attend, _kv4, _q


@pytest.mark.parametrize("rows", [1, 9, 40])
@pytest.mark.parametrize("dtype", [sd.SD_BF16, sd.SD_F32])
def test_contexts_whose_tiles_would_pass_32_bits_are_refused(rows, dtype):
    n = ctypes.c_size_t(0)
    size = lambda length: sd.lib().sd_kv4_attention_workspace_size(  # noqa: E731
        ctypes.byref(_q(max_q_rows=rows, max_kv_len=length)), ctypes.byref(_kv4(dtype=dtype)), 2,
        ctypes.byref(n))
    assert size(1 << 30) == sd.SD_OK
    for length in ((1 << 30) + 1, 2**31 - 1):
        assert size(length) == sd.SD_ERR_INVALID_ARG
        assert _attend(q=_q(max_q_rows=rows, max_kv_len=length),
                       kv=_kv4(dtype=dtype)) == sd.SD_ERR_INVALID_ARG
