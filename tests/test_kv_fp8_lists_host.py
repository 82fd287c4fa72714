"""Lists that the calls around a cache in 8 bits read and write: what the host refuses (no GPU)."""
import ctypes

import pytest

import selective_state_space_mamba2_gb300 as ssd
from selective_state_space_mamba2_gb300 import _binding as B
from tests.test_kv_fp8_host import _commit


@pytest.fixture(scope="module")
def lib():
    ssd.build()
    return ssd.lib()


# two requests, a table of 4 columns at 0x50000 (32 bytes), paths of 3 at 0x60000 (24 bytes)
@pytest.mark.parametrize("out", [0x50000, 0x50000 - 4, 0x50000 + 28, 0x60000, 0x60000 - 4, 0x60000 + 20])
def test_commit_contexts_apart_from_table_and_path(lib, out):
    """Other CTAs read both while the new contexts are written."""
    assert lib.kv_commit_tokens_fp8(ctypes.byref(_commit(context_out=out)), None) == B.SSD_ERR_INVALID_ARG
