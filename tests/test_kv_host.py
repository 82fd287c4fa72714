"""Host-side refusals of the attention-side calls (no GPU): every argument check returns before anything is launched, and
the binding refuses wrong shapes, types and host tensors."""
import ctypes
import os

import pytest
import torch

import selective_state_space_mamba2_gb300 as ssd
from selective_state_space_mamba2_gb300 import _binding as B


@pytest.fixture(scope="module")
def lib():
    ssd.build()
    return ssd.lib()


def _make(cls, sizes, pointers, over):
    a = cls()
    for k, v in sizes.items():
        setattr(a, k, v)
    for i, f in enumerate(pointers):
        setattr(a, f, 0x10000 * (i + 1))
    for k, v in over.items():
        setattr(a, k, v)
    return a


def _tables(**over):
    return _make(B.TablesArgs, dict(num_reqs=2, block_size=16, table_cols=4, free_capacity=8, max_tokens=10,
                                    num_blocks=9, null_block_id=0),
                 ("context_lens", "new_lens", "reserved_lens", "block_table", "free_ring", "ring_in", "ring_out",
                  "cu_seqlens", "seq_lens", "reserved_out", "slots", "positions", "token_req"), over)


@pytest.mark.parametrize("over", [dict(num_reqs=-1), dict(block_size=0), dict(max_tokens=-1), dict(table_cols=-1),
                                  dict(block_size=1 << 16, num_blocks=1 << 15), dict(ring_in=None),
                                  dict(ring_out=0x60000), dict(reserved_out=0x30000), dict(seq_lens=0x10000),
                                  dict(cu_seqlens=0x20000), dict(slots=0x50000), dict(context_lens=None),
                                  dict(block_table=None), dict(free_ring=None), dict(slots=None)])
def test_tables_refusals(lib, over):
    assert lib.kv_block_tables(ctypes.byref(_tables(**over)), None) == B.SSD_ERR_INVALID_ARG


def _qk(**over):
    return _make(B.QkArgs, dict(total_tokens=3, nheads=4, kv_heads=2, headdim=64, rotary_dim=64, max_position=10,
                                dtype=B.SSD_BF16, block_size=16, num_blocks=4, eps=1e-6, q_stride=512, k_stride=512,
                                v_stride=512, cache_block_stride=2048),
                 ("q", "k", "v", "q_weight", "k_weight", "cos_sin", "positions", "slots", "q_out", "k_out", "k_cache",
                  "v_cache"), over)


@pytest.mark.parametrize("over", [
    dict(total_tokens=-1), dict(nheads=3), dict(headdim=60), dict(headdim=264), dict(dtype=5), dict(rotary_dim=63),
    dict(rotary_dim=66), dict(rotary_dim=-2), dict(eps=float("nan")), dict(eps=-1.0), dict(q_stride=255),
    dict(q_stride=516), dict(k_stride=100), dict(q=0x10008), dict(q_out=None), dict(q_out=0x10004), dict(cos_sin=None),
    dict(positions=None), dict(v_cache=None), dict(slots=None), dict(v=None), dict(block_size=0),
    dict(cache_block_stride=2040), dict(num_blocks=1 << 28), dict(q_out=0x10000)])
def test_qk_refusals(lib, over):
    """q_out = q is refused where q is not dense (its rows would be overwritten before they are read)."""
    assert lib.kv_qk_norm_rope(ctypes.byref(_qk(**over)), None) == B.SSD_ERR_INVALID_ARG


def _attn(**over):
    return _make(B.AttentionArgs, dict(total_tokens=5, num_seqs=2, nheads=8, kv_heads=2, headdim=128, dtype=B.SSD_BF16,
                                       block_size=16, num_blocks=9, table_cols=4, max_new_tokens=3, mask_words=1,
                                       scale=0.1, q_stride=1024, k_stride=256, v_stride=256, cache_block_stride=4096),
                 ("q", "k_new", "v_new", "k_cache", "v_cache", "cu_seqlens", "context_lens", "block_table", "tree_mask",
                  "out", "lse"), over)


@pytest.mark.parametrize("over", [
    dict(total_tokens=-1), dict(num_seqs=-1), dict(nheads=7), dict(headdim=100), dict(headdim=264), dict(dtype=2),
    dict(block_size=0), dict(num_blocks=0), dict(table_cols=-1), dict(mask_words=0), dict(scale=float("inf")),
    dict(scale=float("nan")), dict(q_stride=1000), dict(k_stride=255), dict(v_stride=257), dict(cache_block_stride=4000),
    dict(wait_limit_cycles=-1), dict(block_size=1 << 20, num_blocks=1 << 12), dict(table_cols=1 << 28)])
@pytest.mark.parametrize("dtype", [B.SSD_BF16, B.SSD_F32])
def test_attention_refusals(lib, over, dtype):
    a = _attn(**{"dtype": dtype, **over})
    assert lib.kv_tree_attention_workspace_size(ctypes.byref(a)) == 0
    assert lib.kv_tree_attention(ctypes.byref(a), ctypes.c_void_p(0x100000), 1 << 40, None) == B.SSD_ERR_INVALID_ARG


@pytest.mark.parametrize("over", [dict(q=None), dict(q=0x10002), dict(k_new=0x10008), dict(out=None), dict(out=0x10008),
                                  dict(cu_seqlens=None), dict(block_table=None), dict(v_cache=None), dict(lse=0x10002)])
def test_attention_pointer_refusals(lib, over):
    a = _attn(**over)
    assert lib.kv_tree_attention(ctypes.byref(a), ctypes.c_void_p(0x100000), 1 << 40, None) == B.SSD_ERR_INVALID_ARG


@pytest.mark.parametrize("dtype,headdim", [(B.SSD_BF16, 128), (B.SSD_F32, 64)])
def test_attention_workspace_is_checked(lib, dtype, headdim):
    a = _attn(dtype=dtype, headdim=headdim)
    need = lib.kv_tree_attention_workspace_size(ctypes.byref(a))
    assert need > 0
    for ws, size in ((None, need), (0x100000, need - 1), (0x100010, need)):
        assert lib.kv_tree_attention(ctypes.byref(a), ctypes.c_void_p(ws), size, None) == B.SSD_ERR_WORKSPACE


def _commit(**over):
    return _make(B.CommitArgs, dict(total_tokens=5, num_seqs=2, kv_heads=2, headdim=64, dtype=B.SSD_BF16, block_size=16,
                                    num_blocks=4, max_path=2, k_stride=128, v_stride=128, cache_block_stride=2048),
                 ("k_new", "v_new", "slots", "cu_seqlens", "path", "path_lens", "context_lens", "context_out", "k_cache",
                  "v_cache"), over)


@pytest.mark.parametrize("over", [
    dict(total_tokens=-1), dict(headdim=3), dict(kv_heads=0), dict(dtype=9), dict(k_stride=127), dict(v_stride=132),
    dict(max_path=0), dict(path=None), dict(path_lens=None), dict(context_out=None), dict(cu_seqlens=None),
    dict(slots=None), dict(k_cache=0x10008), dict(v_new=None), dict(cache_block_stride=2000), dict(block_size=0),
    dict(num_seqs=1 << 30)])
def test_commit_refusals(lib, over):
    assert lib.kv_commit_tokens(ctypes.byref(_commit(**over)), None) == B.SSD_ERR_INVALID_ARG


def test_empty_calls_are_no_ops(lib):
    assert lib.kv_qk_norm_rope(ctypes.byref(_qk(total_tokens=0)), None) == B.SSD_OK
    assert lib.kv_tree_attention(ctypes.byref(_attn(total_tokens=0)), None, 0, None) == B.SSD_OK
    assert lib.kv_tree_attention(ctypes.byref(_attn(num_seqs=0)), None, 0, None) == B.SSD_OK
    assert lib.kv_commit_tokens(ctypes.byref(_commit(total_tokens=0, num_seqs=0)), None) == B.SSD_OK
    for fn in ("kv_block_tables", "kv_qk_norm_rope", "kv_commit_tokens"):
        assert getattr(lib, fn)(None, None) == B.SSD_ERR_INVALID_ARG
    assert lib.kv_tree_attention(None, None, 0, None) == B.SSD_ERR_INVALID_ARG


def test_binding_refuses_host_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(2, 2, 64)
    kc = torch.zeros(2, 4, 2, 64)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ssd.kv_block_tables(i, i, i, torch.zeros(2, 3, dtype=torch.int32), i, i, 16, 4, 5)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ssd.kv_qk_norm_rope(x, x)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ssd.kv_tree_attention(x, x, x, kc, kc, torch.zeros(2, dtype=torch.int32), i[:1], i[:1].view(1, 1), 2)
    with pytest.raises(ValueError, match="CUDA tensor"):
        ssd.kv_commit_tokens(x, x, kc, kc, i)


def test_no_load_goes_to_several_ctas():
    """One library serves every rank of a run on several GPUs, and the caller's pointers say whose memory is read: the kernels
    hold no multicast load, and no CTA's shared memory is written by another's copies."""
    src = os.path.join(os.path.dirname(os.path.abspath(ssd.__file__)), "csrc")
    for name in sorted(os.listdir(src)):
        with open(os.path.join(src, name)) as f:
            assert "multicast" not in f.read(), name


def test_tensors_of_two_devices_are_refused():
    """The check of every tensor's device, on indices; a call after a refused one starts anew."""
    calls = B._kv()
    assert calls.device_of_call(0, 0) == 0
    for a, b in ((0, 1), (3, 0)):
        with pytest.raises(ValueError, match="second is on cuda:%d, other arguments are on cuda:%d" % (b, a)):
            calls.device_of_call(a, b)
    assert calls.device_of_call(1, 1) == 1


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,blocks", [(1, 5), (3, 1), (1, 1), (3, 5)])
def test_workspace_size_of_single_rows_and_blocks(lib, dtype, T, blocks):
    """The stride of a dimension of one entry says nothing: the size is that of the same call with dense tensors."""
    H, G, D, b = 4, 2, 64, 16

    def made(n, *row, odd):
        return torch.empty(row[0], 1, *row[1:], dtype=dtype).transpose(0, 1) if odd and n == 1 else torch.empty(n, *row, dtype=dtype)

    def size(odd):
        q, k, v, kc, vc = (made(n, *row, odd=odd) for n, row in
                           ((T, (H, D)), (T, (G, D)), (T, (G, D)), (blocks, (b, G, D)), (blocks, (b, G, D))))
        a = ssd.attention_args(q, k, v, kc, vc, torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                               torch.zeros(1, 3, dtype=torch.int32), torch.empty(T, H, D, dtype=dtype), T)
        return ssd.kv_tree_attention_workspace_size(a)

    assert size(True) == size(False) > 0


def test_marshalling_module_is_rebuilt_for_another_torch(lib, monkeypatch):
    """Its object is kept for the torch and the interpreter it was compiled against, and for no other."""
    from selective_state_space_mamba2_gb300 import _build

    class Started(Exception):
        pass

    def run(*args, **kwargs):
        raise Started

    monkeypatch.setattr(_build.subprocess, "run", run)
    _build._compile_calls()  # nothing to do
    monkeypatch.setattr(torch, "__version__", torch.__version__ + "x")
    with pytest.raises(Started):
        _build._compile_calls()


def test_commit_of_paths_without_requests_is_a_no_op(lib):
    """Tensors of no elements have no pointers; without requests, paths say that nothing is copied."""
    none = dict(num_seqs=0, path=None, path_lens=None, context_lens=None, context_out=None)
    assert lib.kv_commit_tokens(ctypes.byref(_commit(**none)), None) == B.SSD_OK
    assert lib.kv_commit_tokens(ctypes.byref(_commit(total_tokens=0, **none)), None) == B.SSD_OK
