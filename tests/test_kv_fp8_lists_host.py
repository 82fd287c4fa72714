"""Lists that the calls around a cache in 8 bits read and write: what the host refuses (no GPU)."""
import ctypes

import pytest

import selective_state_space_mamba2_gb300 as ssd
from selective_state_space_mamba2_gb300 import _binding as B
from tests.test_kv_fp8_host import _commit, _read, _verify
from tests.test_kv_host import _attn


@pytest.fixture(scope="module")
def lib():
    ssd.build()
    return ssd.lib()


# two requests, a table of 4 columns at 0x50000 (32 bytes), paths of 3 at 0x60000 (24 bytes)
@pytest.mark.parametrize("out", [0x50000, 0x50000 - 4, 0x50000 + 28, 0x60000, 0x60000 - 4, 0x60000 + 20])
def test_commit_contexts_apart_from_table_and_path(lib, out):
    """Other CTAs read both while the new contexts are written."""
    assert lib.kv_commit_tokens_fp8(ctypes.byref(_commit(context_out=out)), None) == B.SSD_ERR_INVALID_ARG


@pytest.mark.parametrize("fn,make,name", [
    *(("kv_commit_tokens_fp8", _commit, n) for n in ("cu_seqlens", "context_lens", "path", "path_lens", "context_out", "block_table", "err_word")),
    *(("kv_read_tokens_fp8", _read, n) for n in ("cu_seqlens", "starts", "block_table", "err_word")),
    *(("kv_verify_tokens", _verify, n) for n in ("cu_seqlens", "tokens", "parents", "uniform", "path", "path_lens", "accepted", "next_tokens", "err_word"))])
def test_lists_off_their_alignment(lib, fn, make, name):
    for off in (1, 2, 3):
        a = make(**{name: 0xF00000 + off})
        assert getattr(lib, fn)(ctypes.byref(a), None) == B.SSD_ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["cu_seqlens", "context_lens", "block_table", "err_word", "lse", "tree_mask"])
def test_attention_lists_off_their_alignment(lib, name):
    good = _attn(cache_block_stride=16 * 2 * 128)
    need = lib.kv_tree_attention_fp8_workspace_size(ctypes.byref(good))
    a = _attn(cache_block_stride=16 * 2 * 128, **{name: 0xF00002})
    assert lib.kv_tree_attention_fp8(ctypes.byref(a), 0x1000, 0x2000, 0x100000, need, None) == B.SSD_ERR_INVALID_ARG
