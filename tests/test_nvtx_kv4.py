"""The optional NVTX build (-DSD_NVTX) of the cache appends and 4-bit attention compiles."""
import pytest

from .test_nvtx_build import NVCC
from . import test_nvtx_build


@pytest.mark.skipif(not NVCC, reason="nvcc not available")
def test_kv4_entry_points_compile_with_nvtx_ranges(tmp_path):
    test_nvtx_build.test_entry_points_compile_with_nvtx_ranges("kv4_api.cu", tmp_path)
